// hc_post_bwd.cu -- gradients of the expansion y_k = post_k out + sum_j comb_jk r_j.
//
// With G the gradient of y, per token:
//   dout      = sum_k post_k G_k                  (over channels: a vector)
//   dpost_k   = <out, G_k>,  dcomb_jk = <r_j, G_k>    (sums over channels)
//   dres_j    = sum_k comb_jk G_k                 (a vector, when wanted)
// One pass: each of G, out and r is read once (out and r in bf16 or as kept in
// 8 bits), HC * (HC + 1) running sums stay in registers until the token's end.
// It is an HBM stream with 2 + HC (+ HC) FMAs per stream element: 16,384 tokens of
// 4 x 5120, out and r in 8 bits (1.27 GB), 217 us, 5.9 TB/s; in bf16 (1.68 GB) 256 us, 6.6
// TB/s; with dres 323 and 396 us, 6.0 and 5.9 TB/s.  4,096 of 8 x 5120 in bf16 (757 MB) 139
// us, 5.4 TB/s; in 8 bits (575 MB) 144 us, 4.0 TB/s; with dres 249 and 262 us, 4.4 and 3.5
// TB/s, where the sums take 255 registers and one block is on an SM.
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

// W channels of a bf16 row, and of a kept one.
template <int W>
struct Vec;
template <>
struct Vec<8> {
    using T = uint4;
    static __device__ __forceinline__ void unpack(const T &v, float f[8]) { unpack8(v, f); }
    static __device__ __forceinline__ T pack(const float f[8]) { return pack8(f); }
};
template <>
struct Vec<4> {
    using T = uint2;
    static __device__ __forceinline__ void unpack(const T &v, float f[4]) {
        f[0] = bf16lo(v.x), f[1] = bf16hi(v.x), f[2] = bf16lo(v.y), f[3] = bf16hi(v.y);
    }
    static __device__ __forceinline__ T pack(const float f[4]) {
        return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    }
};
template <bool K8, int W>
struct KeptPart {
    typename Vec<W>::T v;
    __device__ __forceinline__ void load(const Kept &k, int64_t row, int64_t nv, int64_t, int64_t i) {
        v = __ldcs(static_cast<const typename Vec<W>::T *>(k.data) + row * nv + i);
    }
    __device__ __forceinline__ void values(float f[W]) const { Vec<W>::unpack(v, f); }
};
template <>
struct KeptPart<true, 8> : KeptVec<true> {};
template <>
struct KeptPart<true, 4> {
    uint32_t c, b;
    __device__ __forceinline__ void load(const Kept &k, int64_t row, int64_t nv, int64_t nblk,
                                         int64_t i) {
        c = __ldcs(static_cast<const uint32_t *>(k.data) + row * nv + i);
        b = __ldg(k.scales + row * nblk + (i >> 3));
    }
    __device__ __forceinline__ void values(float f[4]) const {
        const float s = kept_scale(b);
        e4m3x4_to_float(c, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] *= s;
    }
};

constexpr __host__ __device__ int part_width(int hc, bool dres) { return hc == 8 && dres ? 4 : 8; }

// 2^lg lanes share a token (32 at least): one warp, or several whose sums
// meet in shared memory; 256 threads hold 256 >> lg tokens.  A lane takes W
// channels at a time: 8, but 4 at hc = 8 where dres is wanted too, with which and
// the 72 sums the registers go no further (4,096 tokens of 8 x 5120 in bf16: 252
// us, with 8 channels 327; without dres 140 us, with 4 channels 150).
//
// The FMAs are two wide over neighbouring k (fma.rn.f32x2): the running sums
// of k and k+1 are one 64-bit register, so the packing costs no register and
// no instruction, and comb's and post's pairs are loaded as they lie.
template <int HC, bool R8, bool O8, bool DRES>
__global__ void __launch_bounds__(256, HC == 4 ? 2 : 1)
    k_post_backward(int64_t n, int64_t d, int64_t nblk, int lg, const uint16_t *g0, Kept out,
                    Kept res, const float *__restrict__ post, const float *__restrict__ comb,
                    uint16_t *__restrict__ dout0, float *__restrict__ dpost,
                    float *__restrict__ dcomb, uint16_t *dres0) {
    constexpr int KP = HC / 2, NS = HC * (HC + 1), W = part_width(HC, DRES);
    using V = Vec<W>;
    __shared__ float red[8][NS];
    griddep_wait_then_release();
    const auto *g = reinterpret_cast<const typename V::T *>(g0);
    auto *dout = reinterpret_cast<typename V::T *>(dout0);
    auto *dres = reinterpret_cast<typename V::T *>(dres0);
    const int64_t nv = d / W;
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
            for (int64_t v = l; v < nv; v += lanes) {
                typename V::T gv[HC];
                KeptPart<R8, W> rv[HC];
                KeptPart<O8, W> ov;
#pragma unroll
                for (int k = 0; k < HC; ++k) gv[k] = __ldcs(g + (t * HC + k) * nv + v);
#pragma unroll
                for (int j = 0; j < HC; ++j) rv[j].load(res, t * HC + j, nv, nblk, v);
                ov.load(out, t, nv, nblk, v);
                uint64_t gp[KP][W];
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    float a[W], b[W];
                    V::unpack(gv[2 * p], a);
                    V::unpack(gv[2 * p + 1], b);
#pragma unroll
                    for (int e = 0; e < W; ++e) gp[p][e] = pack2(a[e], b[e]);
                }
                float f[W], s[W];
                {
                    uint64_t pk[KP];
#pragma unroll
                    for (int p = 0; p < KP; ++p)
                        pk[p] = __ldg(reinterpret_cast<const uint64_t *>(post + t * HC) + p);
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        uint64_t sum = fmul2(pk[0], gp[0][e]);
#pragma unroll
                        for (int p = 1; p < KP; ++p) ffma2(sum, pk[p], gp[p][e]);
                        s[e] = sum2(sum);
                    }
                    __stcs(dout + t * nv + v, V::pack(s));
                }
                ov.values(f);
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    const uint64_t fe = pack2(f[e], f[e]);
#pragma unroll
                    for (int p = 0; p < KP; ++p) ffma2(acc[HC][p], fe, gp[p][e]);
                }
#pragma unroll
                for (int j = 0; j < HC; ++j) {
                    rv[j].values(f);
#pragma unroll
                    for (int e = 0; e < W; ++e) {
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
                        for (int e = 0; e < W; ++e) {
                            uint64_t sum = fmul2(c[0], gp[0][e]);
#pragma unroll
                            for (int p = 1; p < KP; ++p) ffma2(sum, c[p], gp[p][e]);
                            s[e] = sum2(sum);
                        }
                        __stcs(dres + (t * HC + j) * nv + v, V::pack(s));
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
cudaError_t launch(int64_t n, int64_t d, const uint16_t *g, const Kept &out, const Kept &res,
                   const float *post, const float *comb, uint16_t *dout, float *dpost,
                   float *dcomb, uint16_t *dres, const DeviceInfo &di, cudaStream_t s) {
    const int64_t nv = d / part_width(HC, dres != nullptr);
    // a warp per token where the tokens fill the GPU, else more of them, so
    // long as each lane keeps a vector of its own
    int lg = 5;
    while (lg < 8 && (2 << lg) <= nv && (n >> (8 - lg)) < (int64_t)di.sms * 4) ++lg;
    const int64_t want = (n + (256 >> lg) - 1) / (256 >> lg), cap = (int64_t)di.sms * 64;
    const dim3 grid((unsigned)(want < cap ? want : cap));
    auto *kernel = dres != nullptr ? &k_post_backward<HC, R8, O8, true>
                                   : &k_post_backward<HC, R8, O8, false>;
    return launch_overlapped(kernel, grid, dim3(256), 0, s, n, d, kept_blocks(d), lg, g, out, res,
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
    return fn(n, d, g, out, res, post, comb, dout, dpost, dcomb, dres, di, s);
}

}  // namespace hc
