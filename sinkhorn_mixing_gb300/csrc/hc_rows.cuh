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

// The same in pairs, for the two-wide FMAs (fma.rn.f32x2 and its like): half the
// instructions of the sums and products, which is what bounds a row's gradients.
template <int DT>
__device__ __forceinline__ void row_pairs(const uint4 &v, uint64_t p[RowVec<DT>::E / 2]) {
    if (DT == HC_BF16) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < RowVec<DT>::E / 2; ++i) p[i] = bf16x2_to_f32x2(w[i]);
    } else {
        float f[RowVec<DT>::E];
        RowVec<DT>::get(v, f);
#pragma unroll
        for (int i = 0; i < RowVec<DT>::E / 2; ++i) p[i] = pack2(f[2 * i], f[2 * i + 1]);
    }
}
template <int DT>
__device__ __forceinline__ uint4 row_from_pairs(const uint64_t p[RowVec<DT>::E / 2]) {
    float f[RowVec<DT>::E];
#pragma unroll
    for (int i = 0; i < RowVec<DT>::E / 2; ++i) unpack2(p[i], f[2 * i], f[2 * i + 1]);
    return RowVec<DT>::set(f);
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t ffma2_of(uint64_t a, uint64_t b, uint64_t c) {  // a b + c
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

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

// Sums a[0..NS) over the warp, NS = 1, 2 or 4; the sum that is returned to a lane is
// number `which`.  Each step halves what a lane carries, so four sums take 6
// shuffles, not 20.
template <int NS>
__device__ __forceinline__ float warp_sums(const float a[NS], int lane, int &which) {
    static_assert(NS == 1 || NS == 2 || NS == 4, "a power of two");
    float v = a[0];
    which = 0;
    int off = 16;
    if constexpr (NS == 4) {
        const bool up = (lane & 16) != 0, up2 = (lane & 8) != 0;
        const float p = (up ? a[2] : a[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? a[0] : a[2], 16);
        const float q = (up ? a[3] : a[1]) + __shfl_xor_sync(0xFFFFFFFFu, up ? a[1] : a[3], 16);
        v = (up2 ? q : p) + __shfl_xor_sync(0xFFFFFFFFu, up2 ? p : q, 8);
        which = (up ? 2 : 0) + (up2 ? 1 : 0);
        off = 4;
    } else if constexpr (NS == 2) {
        const bool up = (lane & 16) != 0;
        v = (up ? a[1] : a[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? a[0] : a[1], 16);
        which = up ? 1 : 0;
        off = 8;
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1)
        if (k <= off) v += __shfl_xor_sync(0xFFFFFFFFu, v, k);
    return v;
}

// Sums a[0..NS) over the block (whole warps, at most 32) in a fixed order; every
// thread gets them.  `red` holds NS x 32 floats, zeros behind the block's warps
// (clear_red); it is free again after the block's next barrier, so calls that
// take two of them in turn need no other barrier.
template <int NS>
__device__ __forceinline__ void block_sum(float a[NS], float (*red)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int which;
    const float v = warp_sums<NS>(a, lane, which);
    if ((lane & (32 / NS - 1)) == 0) red[which][warp] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) a[i] = 0.0f;
    for (int w = 0; w < warps; w += 4)
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const float4 q = *reinterpret_cast<const float4 *>(&red[i][w]);
            a[i] += (q.x + q.y) + (q.z + q.w);
        }
}

__device__ __forceinline__ void clear_red(float *red, int floats) {
    for (int i = threadIdx.x; i < floats; i += blockDim.x) red[i] = 0.0f;
    __syncthreads();
}

// A row is shared by a group of threads, and a block has several groups: 2^LG lanes
// of a warp where `lg` < 5, a warp (5), or the whole block (kBlockRow).
constexpr int kBlockRow = 6;

// Sums a[0..NS) over the group; `red` as in block_sum.
template <bool BLOCK, int NS>
__device__ __forceinline__ void group_sum(float a[NS], int lg, float (*red)[32]) {
    if (BLOCK) {
        block_sum<NS>(a, red);
    } else {
#pragma unroll
        for (int k = 0; k < 5; ++k)
            if (k < lg)
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    a[i] += __shfl_xor_sync(0xFFFFFFFFu, a[i], 1 << k);
    }
}

// A row's variance comes from one round of sums of (x - p) and (x - p)^2 about a
// number p near its values, the mean of the row's first 16 bytes: with delta =
// mean(x - p), the mean is p + delta and the variance mean((x - p)^2) - delta^2,
// which loses nothing worth naming while delta^2 is at most the variance.  Where it is
// not (or is not finite) the round is repeated about p + delta.  Squares above
// binary32's range make the variance infinite, whatever delta is.
__device__ __forceinline__ float row_variance(float mean_sq, float delta) {
    if (mean_sq == __int_as_float(0x7F800000)) return mean_sq;
    const float var = fmaf(-delta, delta, mean_sq);
    return var < 0.0f ? 0.0f : var;  // a row of one number; NaN stays
}
__device__ __forceinline__ bool row_again(float var, float delta) {
    return !(delta * delta <= var) || var == __int_as_float(0x7F800000);
}
template <int DT>
__device__ __forceinline__ float row_guess(const uint4 &v) {
    float f[RowVec<DT>::E], s = 0.0f;
    RowVec<DT>::get(v, f);
#pragma unroll
    for (int e = 0; e < RowVec<DT>::E; ++e) s += f[e];
    return s * (1.0f / RowVec<DT>::E);
}

// Copies of 16 bytes from global to shared memory, in flight while the thread goes
// on.  A thread waits for and reads what it copied itself, so no barrier is
// needed between the two.
__device__ __forceinline__ void copy16_async(uint4 *dst, const uint4 *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the newest `LEFT` groups of this thread's copies have landed.
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// How a kernel with a ring of copied rows is laid over the GPU.
struct RowPlan {
    int lg;        // a row's group (see kBlockRow)
    int threads;   // of a block
    int groups;    // rows a block has at a time
    size_t ring;   // bytes of shared memory
};

// A row of nv vectors for a kernel whose threads have `vecs` of them at most and copy
// `slots` vectors in all a step, with `stages` steps under way.
inline RowPlan row_plan(int64_t nv, int vecs, int slots, int stages) {
    RowPlan p;
    const int64_t need = (nv + vecs - 1) / vecs;
    if (need <= 32) {
        p.lg = 0;
        while (((int64_t)1 << p.lg) < need) ++p.lg;
        p.threads = 256;
        p.groups = 256 >> p.lg;
    } else {
        p.lg = kBlockRow;
        p.threads = (int)((need + 31) & ~(int64_t)31);
        p.groups = 1;
    }
    p.ring = (size_t)stages * slots * p.threads * 16;
    return p;
}

// Vectors a thread has of a row of nv (max_vecs at most, 4 or 5): those that leave the fewest
// places of a group empty (up to a sixteenth more is taken for more vectors a
// thread, and a group of fewer than four lanes, whose accesses are less than 64
// bytes wide, counts as a tenth empty).  100,000 x 520 in bf16, 65 vectors a row:
// the norm 35.7 us with five a thread, 47.4 with four, two or one.
inline int row_vecs(int64_t nv, int max_threads, int max_vecs) {
    int best = 4;
    float most = 0.0f;
    for (int v : {4, 5, 3, 2, 1}) {
        const RowPlan p = row_plan(nv, v, 1, 1);
        if (p.threads > max_threads || v > max_vecs) continue;
        const int lanes = p.lg == kBlockRow ? p.threads : 1 << p.lg;
        const float fill = (float)nv / (float)(v * lanes) - (lanes < 4 ? 0.1f : 0.0f);
        if (fill > most + 0.0625f) best = v, most = fill;
    }
    return best;
}

// Blocks of `kernel` that an SM holds, from its registers, threads and shared memory.
template <typename K>
int blocks_per_sm(K *kernel, std::atomic<int> &regs, const RowPlan &p) {
    int r = regs.load(std::memory_order_relaxed);
    if (r == 0) {
        cudaFuncAttributes a;
        if (cudaFuncGetAttributes(&a, kernel) != cudaSuccess) return 1;
        r = (a.numRegs + 7) & ~7;
        regs.store(r, std::memory_order_relaxed);
    }
    const int by_regs = 65536 / (r * p.threads), by_threads = 2048 / p.threads;
    const int by_smem = (int)((size_t)(227 * 1024) / (p.ring + 2048));
    int k = by_regs < by_threads ? by_regs : by_threads;
    k = by_smem < k ? by_smem : k;
    return k < 1 ? 1 : k;
}

}  // namespace hc
