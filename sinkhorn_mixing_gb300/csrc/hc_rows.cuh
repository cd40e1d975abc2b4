// hc_rows.cuh -- rows of bf16, fp16 or binary32 numbers in 16-byte vectors, and
// sums over a block.  Shared by the norm's and the embedding's kernels.
#pragma once

#include <cuda_fp16.h>

#include "hc_common.cuh"
#include "hc_rows.h"

namespace hc {

// E channels of a row as they lie in 16 bytes; values are exact in binary32, and
// set() rounds once, to nearest even.
template <int DT>
struct RowVec;
template <>
struct RowVec<HC_BF16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void get(const uint4 &v, float f[E]) { unpack8(v, f); }
    static __device__ __forceinline__ uint4 set(const float f[E]) { return pack8(f); }
};
template <>
struct RowVec<HC_F16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void get(const uint4 &v, float f[E]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = p.x, f[2 * i + 1] = p.y;
        }
    }
    static __device__ __forceinline__ uint4 set(const float f[E]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct RowVec<HC_F32> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void get(const uint4 &v, float f[E]) {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 set(const float f[E]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};

// E binary32 parameters (weight, bias) of vector v; `none` where there are none.
template <int E>
__device__ __forceinline__ void row_params(const float *p, int64_t v, float none, float f[E]) {
#pragma unroll
    for (int q = 0; q < E / 4; ++q) {
        float4 a = make_float4(none, none, none, none);
        if (p != nullptr) a = __ldg(reinterpret_cast<const float4 *>(p) + v * (E / 4) + q);
        f[4 * q] = a.x, f[4 * q + 1] = a.y, f[4 * q + 2] = a.z, f[4 * q + 3] = a.w;
    }
}

// Sums a[0..NS) over the block (whole warps, at most 32) in a fixed order; every
// thread gets them.  `red` holds NS x 32 floats and may be used again after the
// next barrier of the caller's.
template <int NS>
__device__ __forceinline__ void block_sum(float a[NS], float (*red)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < NS; ++i) a[i] += __shfl_xor_sync(0xFFFFFFFFu, a[i], off);
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < NS; ++i) red[i][warp] = a[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) a[i] = lane < warps ? red[i][lane] : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < NS; ++i) a[i] += __shfl_xor_sync(0xFFFFFFFFu, a[i], off);
}

}  // namespace hc
