// hc_rownorm.cu -- the norm of rows: y = (x - mu) r * w + b, r = 1 / sqrt(v + eps),
// v the mean of (x - mu)^2, mu the row's mean (layer norm) or 0 (RMS norm).
#include "hc_rows.cuh"

namespace hc {
namespace {

// Any width: a block a row, the row read once for each sum and once more for the
// output (from L1 or L2 after the first time).
template <int DT, bool CENTER>
__global__ void __launch_bounds__(256)
    k_norm_wide(int64_t rows, int64_t nv, float eps, const uint4 *x0, const float *__restrict__ w,
                const float *__restrict__ b, uint4 *y0) {
    constexpr int E = RowVec<DT>::E;
    __shared__ float red[2][1][32];
    griddep_wait_then_release();
    const float inv_d = 1.0f / (float)(nv * E);
    for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
        const uint4 *x = x0 + t * nv;
        float mu = 0.0f, f[E];
        if (CENTER) {
            float s[1] = {0.0f};
            for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
                RowVec<DT>::get(x[v], f);
#pragma unroll
                for (int e = 0; e < E; ++e) s[0] += f[e];
            }
            block_sum<1>(s, red[0]);
            mu = s[0] * inv_d;
        }
        float q[1] = {0.0f};
        for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
            RowVec<DT>::get(x[v], f);
#pragma unroll
            for (int e = 0; e < E; ++e) q[0] = fmaf(f[e] - mu, f[e] - mu, q[0]);
        }
        block_sum<1>(q, red[1]);
        const float r = rsqrtf(fmaf(q[0], inv_d, eps));
        for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
            float wv[E], bv[E];
            RowVec<DT>::get(x[v], f);
            row_params<E>(w, v, 1.0f, wv);
            row_params<E>(b, v, 0.0f, bv);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = fmaf((f[e] - mu) * r, wv[e], bv[e]);
            y0[t * nv + v] = RowVec<DT>::set(f);
        }
        __syncthreads();  // red is used again by the next row
    }
}

template <int DT, bool CENTER>
cudaError_t launch(const RowNorm &p, const DeviceInfo &di, cudaStream_t s) {
    const int64_t nv = p.d / RowVec<DT>::E, cap = (int64_t)di.sms * 64;
    return launch_overlapped(&k_norm_wide<DT, CENTER>,
                             dim3((unsigned)(p.rows < cap ? p.rows : cap)), dim3(256), 0, s, p.rows,
                             nv, p.eps, static_cast<const uint4 *>(p.x), p.weight, p.bias,
                             static_cast<uint4 *>(p.y));
}

template <int DT>
cudaError_t launch(const RowNorm &p, const DeviceInfo &di, cudaStream_t s) {
    return p.center ? launch<DT, true>(p, di, s) : launch<DT, false>(p, di, s);
}

}  // namespace

cudaError_t launch_norm(const RowNorm &p, const DeviceInfo &di, cudaStream_t s) {
    return p.dtype == HC_BF16  ? launch<HC_BF16>(p, di, s)
           : p.dtype == HC_F16 ? launch<HC_F16>(p, di, s)
                               : launch<HC_F32>(p, di, s);
}

}  // namespace hc
