// hc_pre_bwd.cu -- gradients of hc_mixes_pre (and of the stream that hc_post
// carries past the sublayer).
//
// Per token, with x the stream, F = HC d features, r = (mean x^2 + e)^-1/2, the
// mix numbers m = r x W^T, logits z = m s + b, and G the gradient of the stream
// that hc_post wrote with this call's comb:
//   dpre_j = <dy, x_j>;  dz = the split's gradient from dpre, dpost, dcomb
//   dm = dz s;  du = r dm;  q = -(r^2 / F) sum_i dm_i m_i
//   dx_j = pre_j dy + q x_j + sum_i du_i W_ij + sum_k comb_jk G_k
//   dW = sum over tokens of du x;  ds = sum dz m per group;  db = sum dz
// Nothing of a token's dx is known before its dpre is, which sums over the
// whole row, so the work is cut there: k_mix_backward makes the per-token
// coefficients, k_dx_dw (hc_pre_bwd_main.cu) uses them, k_sum adds the partial
// sums of dW, ds and db in a fixed order.
#include <cuda_fp16.h>

#include "hc_pre_bwd.h"

namespace hc {
namespace {

constexpr int kMaxBlocks = 160 * 3;  // of k_mix_backward: rows of partial sums

template <int HC>
__host__ __device__ constexpr int mix_warps() { return 8 * HC / 32; }
// Blocks on an SM.  (At hc = 4 in bf16 two blocks with four vectors in flight a lane instead of
// two do not pay: the whole call of 4,096 tokens took 157 us against 147.)
template <int HC>
__host__ __device__ constexpr int mix_blocks() { return HC == 4 ? 3 : 2; }

// -------------------------------------------------------- k_mix_backward
// Warps 0-7 sum <dy, x_j> and sum x^2 of up to 8 tokens at a time (2^lg lanes
// a token); mix_warps() more warps meanwhile run the same tokens' split
// forward and backward, which needs neither sum until its end.  HC lanes share
// a token, lane j holding row j of comb: a row step is local, a column step
// sums over the lanes.
//
// The Sinkhorn steps are undone rather than kept: a step leaves its divisors
// (HC numbers) in shared memory, and going back, the matrix before the step is
// the one after it times them.  16,384 tokens of 4 x 5120 in 8 bits (517 MB): 111 us,
// 4.7 TB/s.  For C' = C / den, den = sum C + eps over the
// row (or column):  dC = (dC' - sum dC' C') / den.
// Where a token's record is (Coef): one after the other, or in tiles.
template <int HC>
struct Record {
    using CF = Coef<HC>;
    uint8_t *coef, *tile;
    int r;  // row in the tile, or -1
    __device__ __forceinline__ Record(uint8_t *rec, int64_t t, bool tiled) {
        if (tiled) {
            tile = rec + t / kTileTokens * CF::kTileBytes;
            r = (int)(t % kTileTokens);
            coef = tile + r * CF::kTileCoefBytes;
            tile += kTileTokens * CF::kTileCoefBytes + r % 8 * 16;
        } else {
            coef = rec + t * CF::kBytes;
            tile = coef + CF::kCoefBytes;
            r = -1;
        }
    }
    __device__ __forceinline__ void put16(int i, uint16_t v) const {
        if (r < 0) {
            reinterpret_cast<uint16_t *>(tile)[i] = v;
            return;
        }
        uint8_t *p = tile + (r / 8 * (CF::kK / 8) + i / 8) * 128 + i % 8 * 2;
#pragma unroll
        for (int i = 0; i < CF::kTileRepeats; ++i)
            *reinterpret_cast<uint16_t *>(p + i * kTileTokens * CF::kKBytes) = v;
    }
    __device__ __forceinline__ void put3(int i, uint16_t v) const {
        if (r < 0) {
            reinterpret_cast<uint16_t *>(tile + CF::kKBytes)[i] = v;
            return;
        }
        *reinterpret_cast<uint16_t *>(tile + CF::kTileRepeats * kTileTokens * CF::kKBytes +
                                      (i / 8 * (kTileTokens / 8) + r / 8) * 128 + i % 8 * 2) = v;
    }
};

template <int HC, bool K8>
__global__ void __launch_bounds__(256 + 32 * mix_warps<HC>(), mix_blocks<HC>())
    k_mix_backward(int64_t n, int64_t npad, int64_t nv, int64_t nblk, int lg, int iters, float eps,
                   float norm_eps, float features, const uint4 *__restrict__ dy, Kept x,
                   const float *__restrict__ mixes, const float *__restrict__ scale,
                   const float *__restrict__ base, const float *__restrict__ dpost,
                   const float *__restrict__ dcomb, uint8_t *__restrict__ rec,
                   int tiled, uint8_t *__restrict__ scales, float *__restrict__ partial) {
    using CF = Coef<HC>;
    constexpr int MIX = CF::kMix, MW = mix_warps<HC>(), THREADS = 256 + 32 * MW;
    __shared__ float sums[2][8][HC + 1];
    extern __shared__ float hist[];  // [MW][2 * iters - 1][32]
    griddep_wait_then_release();
    const int tpb = 256 >> lg, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto meet = [] { asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory"); };
    const int64_t groups = (npad + tpb - 1) / tpb;  // npad > n: records of zeros behind

    if (warp < 8) {
        const int lanes = 1 << lg, slot = threadIdx.x >> lg, l = threadIdx.x & (lanes - 1);
        int buf = 0;
        for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x, buf ^= 1) {
            const int64_t t = grp * tpb + slot;
            float acc[HC + 1];
#pragma unroll
            for (int j = 0; j <= HC; ++j) acc[j] = 0.0f;
            if (t < n) {
#pragma unroll 2
                for (int64_t v = l; v < nv; v += lanes) {
                    const uint4 yv = __ldg(dy + t * nv + v);
                    KeptVec<K8> xv[HC];
#pragma unroll
                    for (int j = 0; j < HC; ++j) xv[j].load(x, t * HC + j, nv, nblk, v);
                    const uint64_t y2[4] = {bf16x2_to_f32x2(yv.x), bf16x2_to_f32x2(yv.y),
                                            bf16x2_to_f32x2(yv.z), bf16x2_to_f32x2(yv.w)};
#pragma unroll
                    for (int j = 0; j < HC; ++j) {
                        // A vector lies in one block: its scale comes after its sums (to the
                        // squares twice, as its own square may be infinite, or 0, where theirs
                        // times it is not)
                        uint64_t f[4];
                        const float sc = xv[j].pairs(f);
                        uint64_t dot = fmul2(f[0], y2[0]), sq = fmul2(f[0], f[0]);
#pragma unroll
                        for (int e = 1; e < 4; ++e) {
                            ffma2(dot, f[e], y2[e]);
                            ffma2(sq, f[e], f[e]);
                        }
                        acc[j] = K8 ? fmaf(sc, sum2(dot), acc[j]) : acc[j] + sum2(dot);
                        acc[HC] = K8 ? fmaf(sc, sc * sum2(sq), acc[HC]) : acc[HC] + sum2(sq);
                    }
                }
            }
            if (HC == 4 && K8 && scales != nullptr && t < n) {
                // The scales once more, by slices of 64 channels: k_dx_dw_tma reads a slice of
                // many tokens, and as x has them that would be 2 bytes from each of many rows.
                const int64_t slices = (nv + 7) / 8;
                uint2 *to = reinterpret_cast<uint2 *>(scales) + t % kTileTokens +
                            t / kTileTokens * slices * kTileTokens;
                for (int64_t c = l; c < slices; c += lanes) {
                    uint32_t v[HC];
#pragma unroll
                    for (int j = 0; j < HC; ++j) {
                        const uint8_t *p = x.scales + (t * HC + j) * nblk + 2 * c;
                        v[j] = __ldg(p) | (2 * c + 1 < nblk ? (uint32_t)__ldg(p + 1) << 8 : 0u);
                    }
                    to[c * kTileTokens] = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
                }
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j <= HC; ++j)
#pragma unroll
                for (int off = 16; off > 0; off >>= 1)
                    acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], off);
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j <= HC; ++j) sums[buf][warp][j] = acc[j];
            }
            meet();
        }
        return;
    }

    const int mw = warp - 8, j = lane % HC, slot = mw * (32 / HC) + lane / HC;
    const int steps = 2 * iters - 1;
    float *h = hist + mw * steps * 32;
    const float s0 = __ldg(scale), s1 = __ldg(scale + 1), s2 = __ldg(scale + 2);
    const float b0 = __ldg(base + j), b1 = __ldg(base + HC + j);
    float b2[HC];
#pragma unroll
    for (int k = 0; k < HC; ++k) b2[k] = __ldg(base + 2 * HC + j * HC + k);
    float db0 = 0.0f, db1 = 0.0f, db2[HC], ds0 = 0.0f, ds1 = 0.0f, ds2 = 0.0f;
#pragma unroll
    for (int k = 0; k < HC; ++k) db2[k] = 0.0f;
    // sums v[k] over the HC lanes of a token, in every one of them
    auto over_rows = [](float v[HC]) {
#pragma unroll
        for (int off = 1; off < HC; off <<= 1)
#pragma unroll
            for (int k = 0; k < HC; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], off);
    };

    int buf = 0;
    for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x, buf ^= 1) {
        const bool valid = slot < tpb && grp * tpb + slot < n;
        const int64_t t = valid ? grp * tpb + slot : 0;  // idle lanes follow, and write nothing
        const float *mt = mixes + t * MIX;
        const float m0 = __ldg(mt + j), m1 = __ldg(mt + HC + j);
        float m2[HC], P[HC], C[HC], G[HC], v[HC];
#pragma unroll
        for (int k = 0; k < HC; ++k) m2[k] = __ldg(mt + 2 * HC + j * HC + k);
#pragma unroll
        for (int k = 0; k < HC; ++k) G[k] = __ldg(dcomb + (t * HC + j) * HC + k);
        const float gp = __ldg(dpost + t * HC + j);

        // forward: the softmax P and the Sinkhorn steps, in the order of sinkhorn_comb
#pragma unroll
        for (int k = 0; k < HC; ++k) P[k] = fmaf(m2[k], s2, b2[k]);
        float mx = P[0];
#pragma unroll
        for (int k = 1; k < HC; ++k) mx = fmaxf(mx, P[k]);
#pragma unroll
        for (int k = 0; k < HC; ++k) P[k] = expf(P[k] - mx);
        float inv = rcp_refined(pair_sum(P));
#pragma unroll
        for (int k = 0; k < HC; ++k) {
            C[k] = fmaf(P[k], inv, eps);
            P[k] *= inv;
        }
        __syncwarp();
        for (int i = 0; i < steps; ++i) {
            if (i % 2 == 0) {
#pragma unroll
                for (int k = 0; k < HC; ++k) v[k] = C[k];
                over_rows(v);
                float own = 0.0f;
#pragma unroll
                for (int k = 0; k < HC; ++k) {
                    v[k] += eps;
                    if (k == j) own = v[k];
                    C[k] *= rcp_refined(v[k]);
                }
                h[i * 32 + lane] = own;
            } else {
                const float den = pair_sum(C) + eps;
                inv = rcp_refined(den);
#pragma unroll
                for (int k = 0; k < HC; ++k) C[k] *= inv;
                h[i * 32 + lane] = den;
            }
        }
        __syncwarp();
        const bool pad = slot < tpb && !valid && grp * tpb + slot < npad;
        const Record<HC> to(rec, pad ? grp * tpb + slot : t, tiled != 0);
        float *ct = reinterpret_cast<float *>(to.coef);
        if (valid) {
#pragma unroll
            for (int k = 0; k < HC; ++k) ct[k * HC + j] = C[k];
        }
        // backward through the steps
        for (int i = steps - 1; i >= 0; --i) {
            if (i % 2 == 0) {
#pragma unroll
                for (int k = 0; k < HC; ++k) v[k] = G[k] * C[k];
                over_rows(v);
                const float *dh = h + i * 32 + (lane - j);
#pragma unroll
                for (int k = 0; k < HC; ++k) {
                    const float den = dh[k];
                    G[k] = (G[k] - v[k]) * rcp_refined(den);
                    C[k] *= den;
                }
            } else {
                const float den = h[i * 32 + lane];
#pragma unroll
                for (int k = 0; k < HC; ++k) v[k] = G[k] * C[k];
                const float dot = pair_sum(v);
                inv = rcp_refined(den);
#pragma unroll
                for (int k = 0; k < HC; ++k) {
                    G[k] = (G[k] - dot) * inv;
                    C[k] *= den;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < HC; ++k) v[k] = G[k] * P[k];
        const float dot = pair_sum(v);
#pragma unroll
        for (int k = 0; k < HC; ++k) G[k] = P[k] * (G[k] - dot);  // dz of comb

        // sigmoid(z) and its derivative e / (1+e)^2, e = e^-|z|
        const float z0 = fmaf(m0, s0, b0), e0 = expf(-fabsf(z0)), r0 = rcp_refined(1.0f + e0);
        const float z1 = fmaf(m1, s1, b1), e1 = expf(-fabsf(z1)), r1 = rcp_refined(1.0f + e1);
        const float pre = (z0 >= 0.0f ? r0 : e0 * r0) + eps;
        const float dz1 = 2.0f * gp * (e1 * r1 * r1);

        meet();
        float dpre = 0.0f, ss = 0.0f;
        if (valid) {
            for (int w = 0; w < (1 << lg) / 32; ++w) {
                dpre += sums[buf][slot * ((1 << lg) / 32) + w][j];
                ss += sums[buf][slot * ((1 << lg) / 32) + w][HC];
            }
        }
        const float dz0 = dpre * (e0 * r0 * r0);
        const float r2 = 1.0f / (ss / features + norm_eps), r = sqrtf(r2);
        const float dm0 = dz0 * s0, dm1 = dz1 * s1;
        float c2 = 0.0f;
#pragma unroll
        for (int k = 0; k < HC; ++k) c2 = fmaf(G[k], m2[k], c2);
        float dot_m = fmaf(dm0, m0, fmaf(dm1, m1, c2 * s2));
#pragma unroll
        for (int off = 1; off < HC; off <<= 1)
            dot_m += __shfl_xor_sync(0xFFFFFFFFu, dot_m, off);
        // du, and its forms for the products
        const float du0 = dm0 * r, du1 = dm1 * r, f2 = s2 * r;
        float du2[HC], top = fmaxf(fabsf(du0), fabsf(du1));
#pragma unroll
        for (int k = 0; k < HC; ++k) {
            du2[k] = G[k] * f2;
            top = fmaxf(top, fabsf(du2[k]));
        }
#pragma unroll
        for (int off = 1; off < HC; off <<= 1)
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
        const int ex = min(max((int)(__float_as_uint(top) >> 23), 14), 253);
        const float up = __uint_as_float((uint32_t)(267 - ex) << 23);
        if (valid) {
            ct[CF::kPre + j] = pre;
            if (j < 2) {
                const float v = j == 0 ? -dot_m * r2 / features
                                       : __uint_as_float((uint32_t)(ex - 13) << 23);
                ct[CF::kQ + j] = v;
            }
            auto put = [&](int i, float v) {
                to.put16(i, __half_as_ushort(__float2half_rn(v * up)));
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    const __nv_bfloat16 b = __float2bfloat16_rn(v);
                    const float part = __bfloat162float(b);
                    to.put3(p * MIX + i, __bfloat16_as_ushort(b));
                    // nothing is left of an infinity (inf - inf would be NaN, and dW's sum too)
                    v = fabsf(part) == INFINITY ? 0.0f : v - part;
                }
            };
            put(j, du0);
            put(HC + j, du1);
#pragma unroll
            for (int k = 0; k < HC; ++k) put(2 * HC + j * HC + k, du2[k]);
            for (int i = MIX + j; i < CF::kK; i += HC) to.put16(i, 0);
            for (int i = 3 * MIX + j; i < CF::kParts; i += HC) to.put3(i, 0);
            db0 += dz0, db1 += dz1;
#pragma unroll
            for (int k = 0; k < HC; ++k) db2[k] += G[k];
            ds0 = fmaf(dz0, m0, ds0), ds1 = fmaf(dz1, m1, ds1), ds2 += c2;
        } else if (pad) {
            for (int i = j; i <= CF::kF; i += HC) ct[i] = 0.0f;
            for (int i = j; i < CF::kK; i += HC) to.put16(i, 0);
            for (int i = j; i < CF::kParts; i += HC) to.put3(i, 0);
        }
    }
    // over the tokens of the warp; the scales' sums over the rows as well
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        if (off >= HC) {
            db0 += __shfl_xor_sync(0xFFFFFFFFu, db0, off);
            db1 += __shfl_xor_sync(0xFFFFFFFFu, db1, off);
#pragma unroll
            for (int k = 0; k < HC; ++k) db2[k] += __shfl_xor_sync(0xFFFFFFFFu, db2[k], off);
        }
        ds0 += __shfl_xor_sync(0xFFFFFFFFu, ds0, off);
        ds1 += __shfl_xor_sync(0xFFFFFFFFu, ds1, off);
        ds2 += __shfl_xor_sync(0xFFFFFFFFu, ds2, off);
    }
    float *pt = partial + (int64_t)(blockIdx.x * MW + mw) * (MIX + 4);
    if (lane < HC) {
        pt[j] = db0;
        pt[HC + j] = db1;
#pragma unroll
        for (int k = 0; k < HC; ++k) pt[2 * HC + j * HC + k] = db2[k];
    }
    if (lane == 0) pt[MIX] = ds0, pt[MIX + 1] = ds1, pt[MIX + 2] = ds2;
}

// ----------------------------------------------------------------- k_sum
// dW from the partial sums of the teams that worked on a band, four features a
// thread; behind those blocks, one warp per column of k_mix_backward's partial
// sums.  It adds 9 us to a call at hc = 4 and d = 5120, 21 us at hc = 8.
template <int HC>
__global__ void __launch_bounds__(256) k_sum(Split sp, int64_t d, int per_slice,
                                             const float *__restrict__ dwp,
                                             float *__restrict__ dw, int rows,
                                             const float *__restrict__ mp,
                                             float *__restrict__ dscale,
                                             float *__restrict__ dbase) {
    constexpr int MIX = Coef<HC>::kMix;
    const int CH = sp.channels, FT = HC * CH;
    griddep_wait_then_release();
    const int64_t b = blockIdx.x, dwb = sp.bands * sp.wide * per_slice;
    if (b < dwb) {
        const int64_t s = b / per_slice, band = s / sp.wide, w = s % sp.wide;
        const int e = ((int)(b % per_slice) * 256 + (int)threadIdx.x) * 4;
        const int i = e / FT, m = e % FT;
        const int64_t c = s * CH + m % CH;
        if (i >= MIX || c >= d) return;
        const int64_t c0 = sp.team_of(band * sp.steps), c1 = sp.team_of((band + 1) * sp.steps - 1);
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int64_t p = c0; p <= c1; ++p) {
            const float4 v = *reinterpret_cast<const float4 *>(
                dwp + ((p + band) * sp.wide + w) * MIX * FT + e);
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
        *reinterpret_cast<float4 *>(dw + ((int64_t)i * HC + m / CH) * d + c) = sum;
        return;
    }
    const int lane = threadIdx.x & 31, col = (int)(b - dwb) * 8 + (threadIdx.x >> 5);
    if (col >= MIX + 3) return;
    double a = 0.0;
    for (int r = lane; r < rows; r += 32) a += (double)mp[(int64_t)r * (MIX + 4) + col];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, off);
    if (lane == 0) (col < MIX ? dbase[col] : dscale[col - MIX]) = (float)a;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

// The workspace's parts, in this order.
struct Parts {
    size_t rec, scales, mix, dw, end;
};
template <int HC>
Parts parts(int64_t n, int64_t d) {
    using CF = Coef<HC>;
    Parts p;
    // enough for either kernel that makes dx and dW
    const size_t tiles = (size_t)((n + kTileTokens - 1) / kTileTokens) * CF::kTileBytes;
    const size_t rows = (size_t)n * CF::kBytes;
    p.rec = 0;
    p.scales = up256(HC == 4 && tiles > rows ? tiles : rows);
    p.mix = p.scales + (HC == 4 ? up256((size_t)((n + kTileTokens - 1) / kTileTokens) *
                                        ((d + 63) / 64) * kTileTokens * 8)
                                : 0);
    p.dw = p.mix + up256((size_t)kMaxBlocks * mix_warps<HC>() * (CF::kMix + 4) * 4);
    auto partial = [](const Split &sp) {
        return (size_t)sp.partials() * CF::kMix * HC * sp.channels * 4;
    };
    size_t most = partial(split_dx_dw(n, HC, d, Split::kMaxBlocks));
    if (HC == 4) {
        const size_t other = partial(split_dx_dw_tma(n, d, Split::kMaxBlocks));
        if (other > most) most = other;
    }
    p.end = p.dw + up256(most);
    return p;
}

template <int HC, bool K8>
cudaError_t launch(const PreBackward &p, const DeviceInfo &di, cudaStream_t s) {
    constexpr int MW = mix_warps<HC>(), MIX = Coef<HC>::kMix;
    const int64_t nv = p.d / 8, nblk = kept_blocks(p.d), F = HC * p.d;
    const Parts at = parts<HC>(p.n, p.d);
    MainArgs m;
    m.rec = p.ws + at.rec;
    m.scales = p.ws + at.scales;
    m.dwp = reinterpret_cast<float *>(p.ws + at.dw);
    float *mp = reinterpret_cast<float *>(p.ws + at.mix);
    int lg = 5;
    while (lg < 8 && (2 << lg) <= nv && (p.n >> (8 - lg)) < (int64_t)di.sms * mix_blocks<HC>()) ++lg;
    const bool tiled = dx_dw_tma_takes(p);
    const int64_t npad = tiled ? (p.n + kTileTokens - 1) / kTileTokens * kTileTokens : p.n;
    const int64_t groups = (npad + (256 >> lg) - 1) / (256 >> lg);
    const int64_t most = di.sms * mix_blocks<HC>(), cap = most < kMaxBlocks ? most : kMaxBlocks;
    const int blocks = (int)(groups < cap ? groups : cap);
    const size_t smem = (size_t)MW * (2 * p.iters - 1) * 32 * 4;
    // Asked for whatever this call needs: what a launch may use without asking covers the
    // kernel's static part too.  The limit is the most that any call asks for, not this call's:
    // one with fewer steps on another thread must not lower it before this launch.
    static SmemState state;
    cudaError_t e = allow_smem(state, reinterpret_cast<const void *>(k_mix_backward<HC, K8>),
                               MW * (2 * kBackwardMaxIters - 1) * 32 * 4, di);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(
        k_mix_backward<HC, K8>, dim3(blocks), dim3(256 + 32 * MW), smem, s, p.n, npad, nv, nblk, lg,
        p.iters, p.eps, p.norm_eps, (float)F, reinterpret_cast<const uint4 *>(p.dy), p.x, p.mixes,
        p.scale, p.base, p.dpost, p.dcomb, m.rec, (int)tiled, tiled ? m.scales : nullptr, mp);
    if (e != cudaSuccess) return e;
    const int64_t sms = di.sms < Split::kMaxBlocks ? di.sms : Split::kMaxBlocks;
    m.split = tiled ? split_dx_dw_tma(p.n, p.d, sms) : split_dx_dw(p.n, HC, p.d, sms);
    e = tiled ? launch_dx_dw_tma(p, m, di, s) : launch_dx_dw(p, m, di, s);
    if (e != cudaSuccess) return e;
    const int per_slice = (MIX * HC * m.split.channels / 4 + 255) / 256;
    const int64_t grid = m.split.bands * m.split.wide * per_slice + (MIX + 3 + 7) / 8;
    return launch_overlapped(k_sum<HC>, dim3((unsigned)grid), dim3(256), 0, s, m.split, p.d,
                             per_slice, m.dwp, p.dw, blocks * MW, mp, p.dscale, p.dbase);
}

}  // namespace

size_t pre_backward_bytes(int64_t n, int hc, int64_t d) {
    return hc == 4 ? parts<4>(n, d).end : parts<8>(n, d).end;
}

cudaError_t launch_pre_backward(const PreBackward &p, const DeviceInfo &di, cudaStream_t s) {
    const bool k8 = p.x.scales != nullptr;
    if (p.hc == 4) return k8 ? launch<4, true>(p, di, s) : launch<4, false>(p, di, s);
    return k8 ? launch<8, true>(p, di, s) : launch<8, false>(p, di, s);
}

}  // namespace hc
