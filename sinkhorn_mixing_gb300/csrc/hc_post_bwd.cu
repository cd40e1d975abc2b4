// hc_post_bwd.cu -- gradients of the expansion y_k = post_k out + sum_j comb_jk r_j.
//
// With G the gradient of y, per token:
//   dout      = sum_k post_k G_k                  (over channels: a vector)
//   dpost_k   = <out, G_k>,  dcomb_jk = <r_j, G_k>    (sums over channels)
//   dres_j    = sum_k comb_jk G_k                 (a vector, when wanted)
// One pass: each of G, out and r is read once (out and r in bf16 or as kept in
// 8 bits), HC * (HC + 1) running sums stay in registers until the token's end.
// It is an HBM stream with 2 + HC (+ HC) FMAs per stream element.
#include "hc_kept.cuh"

namespace hc {
namespace {

// Sums a[0..N) over the warp's lanes, each sum ending in one lane (a few of
// them in each): a step halves what a lane carries, so N + 5 shuffles do what a
// butterfly per value does in 5 N.  On return a[0..K) of a lane are sums
// base .. base + count - 1.
template <int N, int OFF>
struct Scatter {
    static constexpr int H = (N + 1) / 2;
    static constexpr int K = Scatter<H, OFF / 2>::K;
    static __device__ __forceinline__ void run(float *a, int lane, int &base, int &count) {
        const bool up = (lane & OFF) != 0;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float lo = a[i], hi = H + i < N ? a[H + i] : 0.0f;
            a[i] = (up ? hi : lo) + __shfl_xor_sync(0xFFFFFFFFu, up ? lo : hi, OFF);
        }
        base += up ? H : 0;
        count = up ? max(count - H, 0) : min(count, H);
        Scatter<H, OFF / 2>::run(a, lane, base, count);
    }
};
template <int N>
struct Scatter<N, 0> {
    static constexpr int K = N;
    static __device__ __forceinline__ void run(float *, int, int &, int &) {}
};

// 2^lg lanes share a token (32 at least): one warp, or several whose sums
// meet in shared memory; 256 threads hold 256 >> lg tokens.
//
// The FMAs are two wide over neighbouring k (fma.rn.f32x2): the running sums
// of k and k+1 are one 64-bit register, so the packing costs no register and
// no instruction, and comb's and post's pairs are loaded as they lie.
template <int HC, bool R8, bool O8, bool DRES>
__global__ void __launch_bounds__(256, HC == 4 ? 2 : 1)
    k_post_backward(int64_t n, int64_t nv, int64_t nblk, int lg, const uint4 *g, Kept out,
                    Kept res, const float *__restrict__ post, const float *__restrict__ comb,
                    uint4 *__restrict__ dout, float *__restrict__ dpost,
                    float *__restrict__ dcomb, uint4 *dres) {
    constexpr int KP = HC / 2, NS = HC * (HC + 1);
    __shared__ float red[8][NS];
    griddep_wait_then_release();
    const int lanes = 1 << lg, slot = threadIdx.x >> lg, l = threadIdx.x & (lanes - 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tpb = 256 >> lg;
    for (int64_t t0 = (int64_t)blockIdx.x * tpb; t0 < n; t0 += (int64_t)gridDim.x * tpb) {
        const int64_t t = t0 + slot;
        uint64_t acc[HC + 1][KP];  // rows j: dcomb; row HC: dpost
#pragma unroll
        for (int j = 0; j <= HC; ++j)
#pragma unroll
            for (int p = 0; p < KP; ++p) acc[j][p] = 0;
        if (t < n) {
            uint64_t pk[KP];
#pragma unroll
            for (int p = 0; p < KP; ++p)
                pk[p] = __ldg(reinterpret_cast<const uint64_t *>(post + t * HC) + p);
            for (int64_t v = l; v < nv; v += lanes) {
                uint4 gv[HC];
                KeptVec<R8> rv[HC];
                KeptVec<O8> ov;
#pragma unroll
                for (int k = 0; k < HC; ++k) gv[k] = ld_stream(g + (t * HC + k) * nv + v);
#pragma unroll
                for (int j = 0; j < HC; ++j) rv[j].load(res, t * HC + j, nv, nblk, v);
                ov.load(out, t, nv, nblk, v);
                uint64_t gp[KP][8];
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    float a[8], b[8];
                    unpack8(gv[2 * p], a);
                    unpack8(gv[2 * p + 1], b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) gp[p][e] = pack2(a[e], b[e]);
                }
                float f[8], s[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    uint64_t d = fmul2(pk[0], gp[0][e]);
#pragma unroll
                    for (int p = 1; p < KP; ++p) ffma2(d, pk[p], gp[p][e]);
                    s[e] = sum2(d);
                }
                st_stream(dout + t * nv + v, pack8(s));
                ov.values(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint64_t fe = pack2(f[e], f[e]);
#pragma unroll
                    for (int p = 0; p < KP; ++p) ffma2(acc[HC][p], fe, gp[p][e]);
                }
#pragma unroll
                for (int j = 0; j < HC; ++j) {
                    rv[j].values(f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint64_t fe = pack2(f[e], f[e]);
#pragma unroll
                        for (int p = 0; p < KP; ++p) ffma2(acc[j][p], fe, gp[p][e]);
                    }
                    if (DRES) {
                        uint64_t c[KP];
#pragma unroll
                        for (int p = 0; p < KP; ++p)
                            c[p] = __ldg(
                                reinterpret_cast<const uint64_t *>(comb + (t * HC + j) * HC) + p);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            uint64_t d = fmul2(c[0], gp[0][e]);
#pragma unroll
                            for (int p = 1; p < KP; ++p) ffma2(d, c[p], gp[p][e]);
                            s[e] = sum2(d);
                        }
                        st_stream(dres + (t * HC + j) * nv + v, pack8(s));
                    }
                }
            }
        }
        float sum[NS];
#pragma unroll
        for (int j = 0; j <= HC; ++j)
#pragma unroll
            for (int p = 0; p < KP; ++p)
                unpack2(acc[j][p], sum[j * HC + 2 * p], sum[j * HC + 2 * p + 1]);
        int base = 0, count = NS;
        Scatter<NS, 16>::run(sum, lane, base, count);
#pragma unroll
        for (int i = 0; i < Scatter<NS, 16>::K; ++i)
            if (i < count) red[warp][base + i] = sum[i];
        __syncthreads();
        if (t < n) {
            for (int i = l; i < NS; i += lanes) {
                float a = 0.0f;
                for (int w = 0; w < (lanes >> 5); ++w) a += red[slot * (lanes >> 5) + w][i];
                if (i < HC * HC)
                    dcomb[t * HC * HC + i] = a;
                else
                    dpost[t * HC + i - HC * HC] = a;
            }
        }
        __syncthreads();
    }
}

template <int HC, bool R8, bool O8>
cudaError_t launch(int64_t n, int64_t d, const uint4 *g, const Kept &out, const Kept &res,
                   const float *post, const float *comb, uint4 *dout, float *dpost, float *dcomb,
                   uint4 *dres, const DeviceInfo &di, cudaStream_t s) {
    const int64_t nv = d / 8;
    // a warp per token where the tokens fill the GPU, else more of them, so
    // long as each lane keeps a vector of its own
    int lg = 5;
    while (lg < 8 && (2 << lg) <= nv && (n >> (8 - lg)) < (int64_t)di.sms * 4) ++lg;
    const int64_t want = (n + (256 >> lg) - 1) / (256 >> lg), cap = (int64_t)di.sms * 64;
    const dim3 grid((unsigned)(want < cap ? want : cap));
    auto *kernel = dres != nullptr ? &k_post_backward<HC, R8, O8, true>
                                   : &k_post_backward<HC, R8, O8, false>;
    return launch_overlapped(kernel, grid, dim3(256), 0, s, n, nv, kept_blocks(d), lg, g, out, res,
                             post, comb, dout, dpost, dcomb, dres);
}

}  // namespace

cudaError_t launch_post_backward(int64_t n, int hc, int64_t d, const uint16_t *g, const Kept &out,
                                 const Kept &res, const float *post, const float *comb,
                                 uint16_t *dout, float *dpost, float *dcomb, uint16_t *dres,
                                 const DeviceInfo &di, cudaStream_t s) {
    const bool r8 = res.scales != nullptr, o8 = out.scales != nullptr;
    auto *fn = hc == 4 ? (r8 ? (o8 ? &launch<4, true, true> : &launch<4, true, false>)
                             : (o8 ? &launch<4, false, true> : &launch<4, false, false>))
                       : (r8 ? (o8 ? &launch<8, true, true> : &launch<8, true, false>)
                             : (o8 ? &launch<8, false, true> : &launch<8, false, false>));
    return fn(n, d, reinterpret_cast<const uint4 *>(g), out, res, post, comb,
              reinterpret_cast<uint4 *>(dout), dpost, dcomb, reinterpret_cast<uint4 *>(dres), di,
              s);
}

}  // namespace hc
