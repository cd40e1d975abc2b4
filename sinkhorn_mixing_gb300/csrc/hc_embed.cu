// hc_embed.cu -- the stream's first value: x[t, j, :] = bf16(scale * table[id_t, :]).
//
// An HBM stream of writes: n * hc * d * 2 bytes, against one table row a token, which
// frequent ids find in the L2.  65,536 tokens of 4 x 5120 from 131,072 bf16 rows (2.89
// GB) 442 us, 6.5 TB/s, 96% of a copy's rate; 4,096 29 us; 64 2.0 us.  A block has 128
// vectors of a token at a time: small blocks, many of them on an SM, and nothing that one
// token's two loads in a row have to wait for in another.
#include "hc_rows.cuh"

namespace hc {
namespace {

// 8 channels of a table row as binary32.
template <int DT>
__device__ __forceinline__ void table_vec(const uint4 *table, int64_t at, float f[8]) {
    constexpr int E = RowVec<DT>::E;
    uint4 v[8 / E];
#pragma unroll
    for (int q = 0; q < 8 / E; ++q) v[q] = __ldg(table + at * (8 / E) + q);
#pragma unroll
    for (int q = 0; q < 8 / E; ++q) RowVec<DT>::get(v[q], f + q * E);
}

template <int DT, typename ID>
__global__ void __launch_bounds__(128)
    k_embed(int64_t n, int hc, int64_t nv, int64_t vocab, float scale, const ID *__restrict__ ids,
            const uint4 *__restrict__ table, uint4 *__restrict__ x) {
    griddep_wait_then_release();
    const int64_t v = (int64_t)blockIdx.y * 128 + threadIdx.x;
    if (v >= nv) return;
    for (int64_t t = blockIdx.x; t < n; t += gridDim.x) {
        const int64_t id = (int64_t)__ldg(ids + t);
        float f[8];
        if (id >= 0 && id < vocab) {
            table_vec<DT>(table, id * nv + v, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= scale;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = 0.0f;
        }
        const uint4 o = pack8(f);
        for (int j = 0; j < hc; ++j) st_stream(x + (t * hc + j) * nv + v, o);
    }
}

template <int DT, typename ID>
cudaError_t launch(const Embed &p, const DeviceInfo &di, cudaStream_t s) {
    const int64_t nv = p.d / 8, cap = (int64_t)di.sms * 64;
    return launch_overlapped(
        &k_embed<DT, ID>,
        dim3((unsigned)(p.n < cap ? p.n : cap), (unsigned)((nv + 127) / 128)), dim3(128), 0, s, p.n,
        p.hc, nv, p.vocab, p.scale, static_cast<const ID *>(p.ids),
        static_cast<const uint4 *>(p.table), reinterpret_cast<uint4 *>(p.x));
}

template <int DT>
cudaError_t launch(const Embed &p, const DeviceInfo &di, cudaStream_t s) {
    return p.id_bytes == 4 ? launch<DT, int32_t>(p, di, s) : launch<DT, int64_t>(p, di, s);
}

}  // namespace

cudaError_t launch_embed(const Embed &p, const DeviceInfo &di, cudaStream_t s) {
    return p.dtype == HC_BF16  ? launch<HC_BF16>(p, di, s)
           : p.dtype == HC_F16 ? launch<HC_F16>(p, di, s)
                               : launch<HC_F32>(p, di, s);
}

}  // namespace hc
