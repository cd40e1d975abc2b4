// hc_pre_bwd.h -- gradients of hc_mixes_pre: sizes shared by its kernels and
// the ABI's workspace rule.
#pragma once

#include "hc_kept.cuh"

namespace hc {

// What the first kernel leaves per token for the second, one record of bytes:
//   coefficients, binary32: comb transposed [k][j] (comb_jk of one k lie
//     together), pre [HC], q, f, padding to a pitch whose rows meet in no bank
//   du16 [kK] fp16: du times a power of two 1/f of the token's own that puts
//     its largest magnitude in [2^13, 2^14), zeros behind (2+HC) HC
//   du3 [kParts] bf16: du = hi + mid + lo, three bf16 numbers (24 bits).
//     HC = 4: [hi | mid | lo | zeros] of 24 each, in 80; HC = 8: 3 x 80.
constexpr int kTileTokens = 32;

template <int HC>
struct Coef {
    static constexpr int kMix = (2 + HC) * HC;
    static constexpr int kPre = HC * HC, kQ = kPre + HC, kF = kQ + 1;  // in floats
    static constexpr int kK = (kMix + 15) / 16 * 16;
    static constexpr int kN = 80;                        // N of one product
    static constexpr int kProducts = HC == 4 ? 1 : 3;
    static constexpr int kParts = kN * kProducts;
    static constexpr int kCoefBytes = HC == 4 ? 112 : 304, kKBytes = kK * 2, kPartBytes = kParts * 2;
    static constexpr int kBytes = kCoefBytes + kKBytes + kPartBytes;
    // For the TMA kernel the records of kTileTokens tokens lie as its shared memory has them:
    // their coefficients, then du16, over and over to 128 rows, and du3 in blocks of 8 x 16 bytes.
    static constexpr int kTileCoefBytes = 96, kTileRepeats = 128 / kTileTokens;
    static constexpr int kTileBytes =
        kTileTokens * (kTileCoefBytes + kTileRepeats * kKBytes + kPartBytes);
    static_assert(kCoefBytes % 16 == 0 && kKBytes % 16 == 0 && kPartBytes % 16 == 0,
                  "16-byte pieces");
    static_assert((kF + 1) * 4 <= kCoefBytes, "coefficients fit");
    static_assert(HC == 4 ? 3 * kMix <= kN : kMix == kN, "three parts fit");
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

// How the work on dx and dW is cut: slices of channels, each walked in steps of
// tokens.  A team of `wide` blocks walks over the same tokens side by side in
// `wide` neighbouring slices (a band), so that what they read and write of a row
// at about the same time is one piece of up to 1 KB: DRAM serves pieces of 128
// bytes at little more than half its rate.  The steps of all bands in a row
// (band-major) are dealt to the teams in equal runs, so every block has the same
// work whatever the shape.  Team c has steps [c * total / teams,
// (c + 1) * total / teams); the partial sums that its block w leaves for band s
// are number (c + s) * wide + w, which no other block has.
struct Split {
    static constexpr int kMaxBlocks = 160;
    int64_t bands, steps, total, teams;
    int channels, wide;
    static Split of(int64_t n, int64_t d, int channels, int tokens, int64_t most) {
        Split s;
        const int64_t slices = (d + channels - 1) / channels;
        s.channels = channels;
        // the widest team that leaves at most 1/16 of its slices empty
        s.wide = 4;
        while (s.wide > 1 && (slices + s.wide - 1) / s.wide * s.wide * 16 > slices * 17) s.wide /= 2;
        s.bands = (slices + s.wide - 1) / s.wide;
        s.steps = (n + tokens - 1) / tokens;
        s.total = s.bands * s.steps;
        s.teams = s.total < most / s.wide ? s.total : most / s.wide;
        return s;
    }
    // (total is below 2^46: n * hc * d is at most 2^58)
    __host__ __device__ int64_t first(int64_t c) const { return c * total / teams; }
    __host__ __device__ int64_t team_of(int64_t step) const {
        return ((step + 1) * teams - 1) / total;
    }
    __host__ __device__ int64_t blocks() const { return teams * wide; }
    __host__ __device__ int64_t partials() const { return (teams + bands) * wide; }
};

struct MainArgs {
    Split split;
    uint8_t *rec;     // per token, or per tile of tokens (Coef)
    uint8_t *scales;  // x's scale bytes for the TMA kernel, [tile][64-channel slice][token][copy][2]
    float *dwp;  // [Split::partials()][mix][hc * channels]
};

constexpr int kBackwardMaxIters = 256;  // Sinkhorn divisors kept in shared memory

size_t pre_backward_bytes(int64_t n, int hc, int64_t d);
Split split_dx_dw(int64_t n, int hc, int64_t d, int64_t most);
Split split_dx_dw_tma(int64_t n, int64_t d, int64_t most);
bool dx_dw_tma_takes(const PreBackward &p);
cudaError_t launch_dx_dw_tma(const PreBackward &p, const MainArgs &m, const DeviceInfo &di,
                             cudaStream_t s);
cudaError_t launch_dx_dw(const PreBackward &p, const MainArgs &m, const DeviceInfo &di,
                         cudaStream_t s);
cudaError_t launch_pre_backward(const PreBackward &p, const DeviceInfo &di, cudaStream_t s);

}  // namespace hc
