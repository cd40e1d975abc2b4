// hc_kept.cuh -- rows kept in 8 bits: the format's arithmetic on the device.
//
// A row of d channels is cut into blocks of 32 (the last one may be shorter).
// A block has one scale byte b, which stands for 2^(b-127), and a channel is an
// e4m3 code c; its value is c * 2^(b-127).  With E and M the biased exponent
// and the mantissa (in [1, 2)) of the block's largest finite magnitude,
//     b = max(1, E - 8 + (M > 1.75)),
// which puts that magnitude over the scale in (224, 448] (448 is the largest
// e4m3 number), so that no finite number saturates, and the scale and its
// reciprocal are normal binary32 numbers.  Scaling by powers of two is exact:
// the one rounding is that to e4m3, to nearest even.  A NaN or an infinity
// becomes the code 0x7F (NaN) and does not take part in the maximum.  A code
// times its scale has 4 significant bits, so it is a bf16 number exactly; the
// largest magnitudes, which would round to 2^128, stay at the number before it
// (240 * 2^120).
#pragma once

#include "hc_common.cuh"
#include "hc_internal.h"

namespace hc {

constexpr int kKeptBlock = 32;  // channels that share a scale
constexpr uint32_t kKeptLastScale = 247;  // of the largest bf16 magnitudes
inline __host__ __device__ int64_t kept_blocks(int64_t d) {
    return (d + kKeptBlock - 1) / kKeptBlock;
}

__device__ __forceinline__ float kept_scale(uint32_t b) { return __uint_as_float(b << 23); }

// Two e4m3 codes (low byte first) as two binary32 numbers, unscaled.
__device__ __forceinline__ void e4m3x2_to_float(uint32_t c, float &lo, float &hi) {
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(h)
        : "r"(c));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\t"
        "cvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
}

__device__ __forceinline__ void e4m3x4_to_float(uint32_t c, float f[4]) {
    e4m3x2_to_float(c & 0xFFFFu, f[0], f[1]);
    e4m3x2_to_float(c >> 16, f[2], f[3]);
}

__device__ __forceinline__ void e4m3x8_to_float(const uint2 &c, float f[8]) {
    e4m3x4_to_float(c.x, f);
    e4m3x4_to_float(c.y, f + 4);
}

// Four numbers as four codes (no number above 448 but NaN).
__device__ __forceinline__ uint32_t float_to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// The scale byte of a block whose largest finite magnitude has the bf16
// pattern `mag` (sign bit clear).
__device__ __forceinline__ uint32_t kept_scale_byte(uint32_t mag) {
    const int b = (int)(mag >> 7) - 8 + ((mag & 0x7Fu) > 0x60u ? 1 : 0);
    return (uint32_t)max(b, 1);
}

// Largest finite magnitude (bf16 pattern) of the 8 channels of `v`; turns its
// infinities into NaNs on the way.
__device__ __forceinline__ uint32_t kept_largest(uint4 &v) {
    uint32_t m = 0;
    uint32_t *w = &v.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t mag = w[i] & 0x7FFF7FFFu;
        const uint32_t bad = __vcmpgeu2(mag, 0x7F807F80u);  // 0xFFFF per half that is not finite
        w[i] |= bad & 0x7FFF7FFFu;
        m = __vmaxu2(m, mag & ~bad);
    }
    return max(m & 0xFFFFu, m >> 16);
}

// The codes of the 8 channels of `v` under the scale byte `byte`.
__device__ __forceinline__ uint2 kept_codes(const uint4 &v, uint32_t byte) {
    const float inv = __uint_as_float((254u - byte) << 23);
    float f[8];
    unpack8(v, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= inv;
    if (byte == kKeptLastScale) {  // 256 * 2^120 is not a bf16 number; NaN stays (ordered compare)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (fabsf(f[e]) > 240.0f) f[e] = copysignf(240.0f, f[e]);
    }
    return make_uint2(float_to_e4m3x4(f[0], f[1], f[2], f[3]),
                      float_to_e4m3x4(f[4], f[5], f[6], f[7]));
}

// Quantises the 8 channels of `v` of one lane: the four lanes of an aligned
// group hold one block.  All lanes of the warp take part; a lane past the
// row's end passes zeros.  Returns the codes; `byte` is the block's scale.
__device__ __forceinline__ uint2 kept_quantise(uint4 v, uint32_t &byte) {
    uint32_t m = kept_largest(v);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    byte = kept_scale_byte(m);
    return kept_codes(v, byte);
}

// A kept tensor's rows, bf16 (K8 = false) or codes and scales (K8 = true), in
// vectors of 8 channels.
struct Kept {
    const void *data;       // [rows, d] bf16 or codes
    const uint8_t *scales;  // [rows, ceil(d / 32)], null for bf16
};

template <bool K8>
struct KeptVec {  // 8 channels as loaded
    uint4 v;
    __device__ __forceinline__ void load(const Kept &k, int64_t row, int64_t nv, int64_t nblk,
                                         int64_t vec) {
        v = __ldcs(static_cast<const uint4 *>(k.data) + row * nv + vec);
    }
    __device__ __forceinline__ void values(float f[8]) const { unpack8(v, f); }
    // the channels in pairs and unscaled; returns their scale
    __device__ __forceinline__ float pairs(uint64_t f[4]) const {
        f[0] = bf16x2_to_f32x2(v.x), f[1] = bf16x2_to_f32x2(v.y);
        f[2] = bf16x2_to_f32x2(v.z), f[3] = bf16x2_to_f32x2(v.w);
        return 1.0f;
    }
};

template <>
struct KeptVec<true> {
    uint2 c;
    uint32_t b;
    __device__ __forceinline__ void load(const Kept &k, int64_t row, int64_t nv, int64_t nblk,
                                         int64_t vec) {
        c = __ldcs(static_cast<const uint2 *>(k.data) + row * nv + vec);
        b = __ldg(k.scales + row * nblk + (vec >> 2));
    }
    __device__ __forceinline__ void values(float f[8]) const {
        const float s = kept_scale(b);
        e4m3x8_to_float(c, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= s;
    }
    __device__ __forceinline__ float pairs(uint64_t f[4]) const {
        float u[8];
        e4m3x8_to_float(c, u);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = pack2(u[2 * e], u[2 * e + 1]);
        return kept_scale(b);
    }
};

// Launchers (hc_kept.cu, hc_post_bwd.cu); arguments are validated before.
cudaError_t launch_checkpoint(int64_t rows, int64_t d, const uint16_t *x, uint8_t *codes,
                              uint8_t *scales, const DeviceInfo &di, cudaStream_t s);
cudaError_t launch_restore(int64_t rows, int64_t d, const Kept &k, uint16_t *x,
                           const DeviceInfo &di, cudaStream_t s);
cudaError_t launch_pre_restore(int64_t n, int hc, int64_t d, const Kept &k, const float *pre,
                               uint16_t *y, const DeviceInfo &di, cudaStream_t s);
cudaError_t launch_post_checkpoint(int64_t n, int hc, int64_t d, const uint16_t *out,
                                   const uint16_t *res, const float *post, const float *comb,
                                   uint16_t *y, uint8_t *codes, uint8_t *scales,
                                   const DeviceInfo &di, cudaStream_t s);
cudaError_t launch_post_backward(int64_t n, int hc, int64_t d, const uint16_t *g, const Kept &out,
                                 const Kept &res, const float *post, const float *comb,
                                 uint16_t *dout, float *dpost, float *dcomb, uint16_t *dres,
                                 const DeviceInfo &di, cudaStream_t s);

// Programmatic dependent launch of a kernel that starts with
// griddep_wait_then_release() (see overlap_launches).
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = overlap_launches() ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) return e;
    return launched();
}

}  // namespace hc
