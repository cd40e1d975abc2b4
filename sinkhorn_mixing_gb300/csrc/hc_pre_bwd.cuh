// hc_pre_bwd.cuh -- device helpers shared by the two kernels that make dx and dW.
#pragma once

#include "hc_ptx.cuh"

namespace hc {
namespace ptx {

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float v[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
        "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
        "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// the values of loads that have been waited for, not to be used before
template <int N>
__device__ __forceinline__ void arrived(float v[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
// The calling thread's products still under way, after which a block may end: they read its shared
// memory and write its TMEM.  `bar` (count 1) has had no arrival, so that the phase that is waited
// for is this commit's whatever other barriers' waits gave up on.
__device__ __forceinline__ void settle_products(uint32_t bar) {
    mma_commit(bar);
    settle_bar(bar, 0);
}
// a binary32 pattern in both halves of a pair
__device__ __forceinline__ uint64_t twice(uint32_t v) {
    return pack2(__uint_as_float(v), __uint_as_float(v));
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return pack_bf16x2(lo, hi);
}
// Shared-memory matrix descriptor without swizzle: blocks of 8 x 16 bytes, `k`
// bytes to the next block along K, `mn` along M or N.
__device__ __forceinline__ uint64_t rows16(uint32_t saddr, uint32_t k, uint32_t mn) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(k >> 4) << 16) |
           ((uint64_t)(mn >> 4) << 32) | ((uint64_t)1 << 46);
}

}  // namespace ptx
}  // namespace hc
