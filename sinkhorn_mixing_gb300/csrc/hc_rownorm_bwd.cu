// hc_rownorm_bwd.cu -- gradients of the norm y = h w + b, h = (x - mu) r.
//
// With g = dy w, per row:
//   dx = r (g - mean(g) [layer norm] - h mean(g h))
// and over the rows dw = sum dy h, db = sum dy.
//
// The sums over rows: every block adds up the rows it has, in registers, and
// leaves one row of partial sums; k_norm_sum adds those up in a fixed order.
#include "hc_rows.cuh"

namespace hc {
namespace {

constexpr int kMaxParts = 304;  // rows of partial sums: two for each of a GB300's 152 SMs

// rows of partial sums at most, by the width
int64_t max_parts(int64_t rows, int64_t d) {
    int64_t m = d <= 16384 ? kMaxParts : (int64_t)kMaxParts * 4096 / d;
    m = m < 1 ? 1 : m;
    return rows < m ? rows : m;
}

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

// Any width, first part: a row's mean, r, mean(g) and mean(g h).
template <int DT, bool CENTER>
__global__ void __launch_bounds__(256)
    k_norm_stats(int64_t rows, int64_t nv, float eps, const uint4 *__restrict__ dy0,
                 const uint4 *__restrict__ x0, const float *__restrict__ w,
                 float4 *__restrict__ stats) {
    constexpr int E = RowVec<DT>::E;
    __shared__ float red[3][2][32];
    griddep_wait_then_release();
    const float inv_d = 1.0f / (float)(nv * E);
    for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
        const uint4 *x = x0 + t * nv, *dy = dy0 + t * nv;
        float mu = 0.0f, f[E], g[E], wv[E];
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
        float c[2] = {0.0f, 0.0f};
        for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
            RowVec<DT>::get(x[v], f);
            RowVec<DT>::get(dy[v], g);
            row_params<E>(w, v, 1.0f, wv);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float ge = g[e] * wv[e];
                c[0] += ge;
                c[1] = fmaf(ge, (f[e] - mu) * r, c[1]);
            }
        }
        block_sum<2>(c, red[2]);
        if (threadIdx.x == 0)
            stats[t] = make_float4(mu, r, CENTER ? c[0] * inv_d : 0.0f, c[1] * inv_d);
        __syncthreads();  // red is used again by the next row
    }
}

// Second part: a block has 128 vectors of a run of rows.
template <int DT>
__global__ void __launch_bounds__(128)
    k_norm_grad(int64_t rows, int64_t nv, int64_t run, const uint4 *dy,
                const uint4 *__restrict__ x, const float *__restrict__ w,
                const float4 *__restrict__ stats, uint4 *dx, float *__restrict__ dw,
                float *__restrict__ db) {
    constexpr int E = RowVec<DT>::E;
    griddep_wait_then_release();
    const int64_t v = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (v >= nv) return;
    const int64_t t0 = (int64_t)blockIdx.y * run, t1 = t0 + run < rows ? t0 + run : rows;
    float wv[E], aw[E], ab[E];
    row_params<E>(w, v, 1.0f, wv);
#pragma unroll
    for (int e = 0; e < E; ++e) aw[e] = ab[e] = 0.0f;
    for (int64_t t = t0; t < t1; ++t) {
        const float4 st = __ldg(stats + t);
        float f[E], g[E];
        RowVec<DT>::get(x[t * nv + v], f);
        RowVec<DT>::get(dy[t * nv + v], g);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float h = (f[e] - st.x) * st.y;
            aw[e] = fmaf(g[e], h, aw[e]);
            ab[e] += g[e];
            f[e] = (fmaf(g[e], wv[e], -st.z) - h * st.w) * st.y;
        }
        dx[t * nv + v] = RowVec<DT>::set(f);
    }
    const int64_t at = ((int64_t)blockIdx.y * nv + v) * (E / 4);
#pragma unroll
    for (int q = 0; q < E / 4; ++q) {
        if (dw != nullptr)
            reinterpret_cast<float4 *>(dw)[at + q] =
                make_float4(aw[4 * q], aw[4 * q + 1], aw[4 * q + 2], aw[4 * q + 3]);
        if (db != nullptr)
            reinterpret_cast<float4 *>(db)[at + q] =
                make_float4(ab[4 * q], ab[4 * q + 1], ab[4 * q + 2], ab[4 * q + 3]);
    }
}

// out[c] = sum over the partial rows of part[p][c]: 8 warps of a block take every
// eighth row of 128 channels, and their sums meet in shared memory.
__global__ void __launch_bounds__(256)
    k_norm_sum(int parts, int64_t d4, const float4 *__restrict__ part_w, float4 *__restrict__ dw,
               const float4 *__restrict__ part_b, float4 *__restrict__ db) {
    __shared__ float4 red[8][32];
    griddep_wait_then_release();
    const float4 *part = blockIdx.y == 0 ? part_w : part_b;
    float4 *out = blockIdx.y == 0 ? dw : db;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (out != nullptr && c < d4) {
#pragma unroll 4
        for (int p = warp; p < parts; p += 8) {
            const float4 v = part[(int64_t)p * d4 + c];
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
    }
    red[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && out != nullptr && c < d4) {
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            const float4 v = red[i][lane];
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
        out[c] = a;
    }
}

template <int DT, bool CENTER>
cudaError_t launch(const RowNormBackward &p, const DeviceInfo &di, cudaStream_t s) {
    const int64_t nv = p.d / RowVec<DT>::E, cap = (int64_t)di.sms * 64;
    const uint4 *dy = static_cast<const uint4 *>(p.dy), *x = static_cast<const uint4 *>(p.x);
    float4 *stats = reinterpret_cast<float4 *>(p.ws);
    const int64_t most = max_parts(p.rows, p.d), run = (p.rows + most - 1) / most;
    const int parts = (int)((p.rows + run - 1) / run);
    float *part_w = reinterpret_cast<float *>(p.ws + align256((size_t)p.rows * 16));
    float *part_b = part_w + (size_t)parts * p.d;
    cudaError_t e = launch_overlapped(&k_norm_stats<DT, CENTER>,
                                      dim3((unsigned)(p.rows < cap ? p.rows : cap)), dim3(256), 0,
                                      s, p.rows, nv, p.eps, dy, x, p.weight, stats);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(&k_norm_grad<DT>, dim3((unsigned)((nv + 127) / 128), (unsigned)parts),
                          dim3(128), 0, s, p.rows, nv, run, dy, x, p.weight,
                          (const float4 *)stats, static_cast<uint4 *>(p.dx),
                          p.dweight ? part_w : nullptr, p.dbias ? part_b : nullptr);
    if (e != cudaSuccess || (p.dweight == nullptr && p.dbias == nullptr)) return e;
    const int64_t d4 = p.d / 4;
    return launch_overlapped(&k_norm_sum, dim3((unsigned)((d4 + 31) / 32), p.dbias ? 2u : 1u),
                             dim3(256), 0, s, parts, d4, (const float4 *)part_w,
                             reinterpret_cast<float4 *>(p.dweight), (const float4 *)part_b,
                             reinterpret_cast<float4 *>(p.dbias));
}

template <int DT>
cudaError_t launch(const RowNormBackward &p, const DeviceInfo &di, cudaStream_t s) {
    return p.center ? launch<DT, true>(p, di, s) : launch<DT, false>(p, di, s);
}

}  // namespace

size_t norm_backward_bytes(int64_t rows, int64_t d) {
    return align256((size_t)rows * 16) + (size_t)max_parts(rows, d) * (size_t)d * 8;
}

cudaError_t launch_norm_backward(const RowNormBackward &p, const DeviceInfo &di, cudaStream_t s) {
    return p.dtype == HC_BF16  ? launch<HC_BF16>(p, di, s)
           : p.dtype == HC_F16 ? launch<HC_F16>(p, di, s)
                               : launch<HC_F32>(p, di, s);
}

}  // namespace hc
