// hc_pre_bwd_main.cu -- dx and dW of hc_mixes_pre's gradient (hc_pre_bwd.cu has
// the formulas), from the per-token coefficients.
//
// Per stream element dx takes HC + 3 FMAs and both products (du W into dx, du^T x
// into dW) another 2 (2+HC) HC: at HC = 4 more than the CUDA cores could do in
// the time the bytes take, so the products run on the tensor cores.
//   du W: its K is the mix count (24 or 80), its result is wanted in registers
//     where the other terms are added: warp-level mma.m16n8k16 on fp16 operands,
//     scaled by powers of two per token (du16) and per slice (W), 11 bits each,
//     which is far below the rounding of dx to bf16.
//   du^T x: its K is the token count, so its result stays for the whole kernel:
//     tcgen05.mma with the sums in TMEM, x^T (exact in bf16) as the M = 128
//     operand and du in three bf16 parts (24 bits) as N; dW keeps binary32's
//     precision.
// A block owns a slice of channels of all copies (512 features), with its part
// of W in shared memory, and walks over tokens in steps (Split); each step's
// tiles come through a two-stage ring of 16-byte asynchronous copies, the next
// step's loads running under this one's arithmetic.
#include <cuda_fp16.h>

#include "hc_pre_bwd.h"
#include "hc_ptx.cuh"

namespace hc {
namespace {

using namespace ptx;

struct Args {
    Split split;
    int64_t n, d, nblk;
    const uint16_t *dy;
    const uint8_t *x, *xs;  // bf16 rows or codes, scales
    const float *w;
    const uint16_t *g;      // may be null
    uint16_t *dx;
    const float *cf;
    const uint16_t *du16, *du3;
    float *dwp;
    unsigned int *err;
};

template <int HC, bool K8>
struct Cfg {
    using CF = Coef<HC>;
    static constexpr int T = Split::tokens(HC), CH = Split::channels(HC), FT = HC * CH;
    static constexpr int MIX = CF::kMix, KS = CF::kK / 16;
    // a warp: 16 tokens, 16 channels, 4 copies; a lane of it 2 tokens, 4 channels
    static constexpr int MT = T / 16, GROUPS = CH / 16, JQ = HC / 4, WARPS = MT * GROUPS * JQ;
    static constexpr int THREADS = 32 * WARPS, MTILES = FT / 128;
    // Row pitches: a token's row is moved on by as many bytes as the lanes of one token read at
    // once, so that the lanes of neighbouring tokens meet in no bank.
    static constexpr int GP = HC * CH * 2 + 32, YP = CH * 2 + 32, XP = HC * CH + 16;
    static constexpr int CP = HC == 4 ? CF::kCf * 4 + 16 : CF::kCf * 4, AP = CF::kK * 2 + 16;
    // x as the M operand: 8 channels x 8 tokens in 128 bytes (channels along 16 bytes), the
    // blocks of a channel group's tokens in a row
    static constexpr int OT = T / 8 * 128, OBYTES = FT / 8 * OT;
    static constexpr int BT = T / 8 * 128, BBYTES = CF::kParts / 8 * BT;
    // stage
    static constexpr int SG = 0, SY = SG + T * GP, SX = SY + T * YP;
    static constexpr int SS = SX + (K8 ? T * XP : OBYTES);  // scales
    static constexpr int SC = SS + (K8 ? T * HC * CH / 32 : 0), SA = SC + T * CP;
    static constexpr int STAGE = (SA + T * AP + 127) / 128 * 128;
    // the block's memory
    static constexpr int BRING = K8 ? 3 : 2;
    static constexpr int OB = 2 * STAGE, OO = OB + BRING * BBYTES;  // du3 ring; x operand (K8)
    static constexpr int OW = OO + (K8 ? OBYTES : 0), WREG = 2 * KS;
    static constexpr int WBYTES = FT / 8 * 32 * WREG * 4;
    static constexpr int OE = OW + WBYTES;                          // barrier, flags, maxima
    static constexpr int SMEM = OE + 256;
    static constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                                      ((uint32_t)(CF::kN >> 3) << 17) | (8u << 24);
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(T * HC * CH / 32 <= THREADS, "a scale byte per thread");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 8 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_wait_all() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
    const uint4 v = lds128(a);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                       __uint_as_float(v.w));
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void mma_f16(float c[4], const uint32_t a[4], uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Shared-memory matrix descriptor without swizzle, the M or N axis along the
// 16-byte rows of 8 x 8 blocks: `mn` bytes to the next 8 of that axis, `k` to
// the next 8 of K.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr, uint32_t k, uint32_t mn) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(k >> 4) << 16) |
           ((uint64_t)(mn >> 4) << 32) | ((uint64_t)1 << 46);
}

template <int HC, bool K8>
__global__ void __launch_bounds__(Cfg<HC, K8>::THREADS, 1) k_dx_dw(Args a) {
    using C = Cfg<HC, K8>;
    using CF = Coef<HC>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = su32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bar = sb + C::OE;
    volatile int *abort = reinterpret_cast<int *>(smem + C::OE + 8);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OE + 12);
    float *maxima = reinterpret_cast<float *>(smem + C::OE + 16);  // per warp

    if (tid == 0) {
        mbar_init(bar, 1);
        *abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         su32(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // lane's place: tokens mt*16 + lane/4 (+ 8), channels cl .. cl+3 of the slice, copies jq*4 ..
    const int mt = warp % C::MT, grp = warp / C::MT % C::GROUPS, jq = warp / (C::MT * C::GROUPS);
    const int tg = lane >> 2, tl = lane & 3, cl = grp * 16 + tl * 4;
    const int64_t F = HC * a.d;
    uint32_t commits = 0;  // products committed to `bar` so far
    auto products_done = [&] {
        return commits == 0 || wait_bar<false>(bar, (commits - 1) & 1, abort, a.err);
    };

    bool started = false;  // has this kernel waited for the one before it
    int64_t step = a.split.first(blockIdx.x);
    const int64_t end = a.split.first(blockIdx.x + 1);
    while (step < end) {
        const int64_t slice = step / a.split.steps;
        const int64_t s0 = step - slice * a.split.steps;
        const int64_t s1 = min(a.split.steps, s0 + (end - step));
        const int64_t ch0 = slice * C::CH;
        const int width = (int)min((int64_t)C::CH, a.d - ch0);

        // ---- the slice of W, in fp16 times a power of two that brings its largest magnitude
        // to [2^13, 2^14), laid out as the products' B fragments
        float top = 0.0f;
        for (int q = tid; q < C::MIX * C::FT; q += C::THREADS) {
            const int i = q / C::FT, m = q % C::FT, c = m % C::CH;
            if (c < width)
                top = fmaxf(top, fabsf(__ldg(a.w + (int64_t)i * F + m / C::CH * a.d + ch0 + c)));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
        if (lane == 0) maxima[warp] = top;
        __syncthreads();
        top = maxima[lane % C::WARPS];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
        const int ex = min(max((int)(__float_as_uint(top) >> 23), 14), 253);
        const float wup = __uint_as_float((uint32_t)(267 - ex) << 23);
        const float wdown = __uint_as_float((uint32_t)(ex - 13) << 23);
        for (int q = tid; q < CF::kK * C::FT; q += C::THREADS) {
            const int i = q / C::FT, m = q % C::FT, j = m / C::CH, c = m % C::CH;
            float v = 0.0f;
            if (i < C::MIX && c < width) v = __ldg(a.w + (int64_t)i * F + j * a.d + ch0 + c);
            // channel 4 t + 2 p + b of its group of 16 is row n = 2 t + b of product p
            const int g = (c >> 2 & 3) * 2 + (c & 1), p = c >> 1 & 1;
            const int k = i & 15, reg = (i >> 4) * 2 + (k >> 3);
            const int nt = (j * C::GROUPS + (c >> 4)) * 2 + p, ln = g * 4 + (k & 7) / 2;
            reinterpret_cast<__half *>(
                smem + C::OW)[((nt * 32 + ln) * C::WREG + reg) * 2 + (k & 1)] =
                __float2half_rn(v * wup);
        }
        if (!started) {
            griddep_wait_then_release();
            started = true;
        }

        // ---- loads of one step's tiles
        auto load = [&](int64_t s, int64_t rel) {
            const uint32_t st = sb + (uint32_t)(s & 1) * C::STAGE;
            const uint32_t bt = sb + C::OB + (uint32_t)(rel % C::BRING) * C::BBYTES;
            const int64_t t0 = s * C::T;
            const int left = (int)min((int64_t)C::T, a.n - t0);
            auto rows = [&](int per, auto place) {
                for (int q = tid; q < C::T * per; q += C::THREADS) place(q / per, q % per);
            };
            if (a.g != nullptr)
                rows(C::FT / 8, [&](int t, int v) {
                    const int k = v / (C::CH / 8), c = v % (C::CH / 8) * 8;
                    const bool in = t < left && c < width;
                    const uint16_t *src = a.g + (t0 + t) * F + k * a.d + ch0 + c;
                    cp16(st + C::SG + t * C::GP + v * 16, in ? src : a.g, in);
                });
            rows(C::CH / 8, [&](int t, int v) {
                const bool in = t < left && v * 8 < width;
                const uint16_t *src = a.dy + (t0 + t) * a.d + ch0 + v * 8;
                cp16(st + C::SY + t * C::YP + v * 16, in ? src : a.dy, in);
            });
            if (!K8) {
                rows(C::FT / 8, [&](int t, int v) {
                    const int j = v / (C::CH / 8), c = v % (C::CH / 8) * 8;
                    const bool in = t < left && c < width;
                    const uint8_t *src = a.x + ((t0 + t) * F + j * a.d + ch0 + c) * 2;
                    cp16(st + C::SX + v * C::OT + t / 8 * 128 + t % 8 * 16, in ? src : a.x, in);
                });
            } else if (a.d % 16 == 0) {
                rows(C::FT / 16, [&](int t, int v) {
                    const int j = v / (C::CH / 16), c = v % (C::CH / 16) * 16;
                    const bool in = t < left && c < width;
                    const uint8_t *src = a.x + (t0 + t) * F + j * a.d + ch0 + c;
                    cp16(st + C::SX + t * C::XP + v * 16, in ? src : a.x, in);
                });
            } else {
                rows(C::FT / 8, [&](int t, int v) {
                    const int j = v / (C::CH / 8), c = v % (C::CH / 8) * 8;
                    const bool in = t < left && c < width;
                    const uint8_t *src = a.x + (t0 + t) * F + j * a.d + ch0 + c;
                    cp8(st + C::SX + t * C::XP + v * 8, in ? src : a.x, in);
                });
            }
            rows(CF::kCf / 4, [&](int t, int v) {
                const bool in = t < left;
                cp16(st + C::SC + t * C::CP + v * 16,
                     in ? a.cf + (t0 + t) * CF::kCf + v * 4 : a.cf, in);
            });
            rows(CF::kK / 8, [&](int t, int v) {
                const bool in = t < left;
                cp16(st + C::SA + t * C::AP + v * 16,
                     in ? a.du16 + (t0 + t) * CF::kK + v * 8 : a.du16, in);
            });
            rows(CF::kParts / 8, [&](int t, int v) {
                const bool in = t < left;
                cp16(bt + v * C::BT + t / 8 * 128 + t % 8 * 16,
                     in ? a.du3 + (t0 + t) * CF::kParts + v * 8 : a.du3, in);
            });
        };
        // the scale byte of (token, copy, block) = tid of step s
        auto load_scale = [&](int64_t s) -> uint32_t {
            constexpr int B = C::CH / 32;
            const int t = tid / (HC * B), j = tid / B % HC, b = tid % B;
            const int64_t tok = s * C::T + t;
            if (!K8 || t >= C::T || tok >= a.n || b * 32 >= width) return 0;
            return __ldg(a.xs + (tok * HC + j) * a.nblk + ch0 / 32 + b);
        };
        auto keep_scale = [&](int64_t s, uint32_t v) {
            if (K8 && tid < C::T * HC * C::CH / 32)
                smem[(s & 1) * C::STAGE + C::SS + tid] = (uint8_t)v;
        };
        // dW += du^T x of the step `rel` of this run: one thread issues
        auto issue = [&](int64_t s, int64_t rel) {
            const uint32_t xo =
                K8 ? sb + C::OO : sb + (uint32_t)(s & 1) * C::STAGE + C::SX;
            const uint32_t bo = sb + C::OB + (uint32_t)(rel % C::BRING) * C::BBYTES;
#pragma unroll
            for (int ks = 0; ks < C::T / 16; ++ks)
#pragma unroll
                for (int m = 0; m < C::MTILES; ++m)
#pragma unroll
                    for (int p = 0; p < CF::kProducts; ++p)
                        mma_bf16(tmem + m * CF::kN,
                                 mn_desc(xo + m * 16 * C::OT + ks * 256, 128, C::OT),
                                 mn_desc(bo + p * (CF::kN / 8) * C::BT + ks * 256, 128, C::BT),
                                 C::IDESC, rel > 0 || ks > 0 || p > 0);
            mma_commit(bar);
        };

        load(s0, 0);
        keep_scale(s0, load_scale(s0));
        for (int64_t s = s0; s < s1; ++s) {
            const int64_t rel = s - s0;
            cp_wait_all();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before();
            __syncthreads();  // step s has landed; all are done with step s - 1
            if (!K8 && rel > 0) products_done();  // of step s - 1, whose x is loaded over
            if (tid == 0 && (!K8 || rel > 0)) {
                tc_fence_after();
                issue(K8 ? s - 1 : s, K8 ? rel - 1 : rel);
            }
            if (!K8 || rel > 0) ++commits;
            uint32_t next_scale = 0;
            if (s + 1 < s1) {
                load(s + 1, rel + 1);
                next_scale = load_scale(s + 1);
            }

            // ---- du W
            const uint32_t st = sb + (uint32_t)(s & 1) * C::STAGE;
            float acc[4][2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][p][e] = 0.0f;
            uint32_t af[C::KS][4];
#pragma unroll
            for (int ks = 0; ks < C::KS; ++ks) {
                const uint32_t ad = st + C::SA + (mt * 16 + (lane & 15)) * C::AP + ks * 32 +
                                    (lane >> 4) * 16;
                asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                             : "=r"(af[ks][0]), "=r"(af[ks][1]), "=r"(af[ks][2]), "=r"(af[ks][3])
                             : "r"(ad));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint32_t wa =
                        sb + C::OW +
                        ((((jq * 4 + j) * C::GROUPS + grp) * 2 + p) * 32 + lane) * C::WREG * 4;
                    if (C::KS == 2) {
                        const uint4 b = lds128(wa);
                        mma_f16(acc[j][p], af[0], b.x, b.y);
                        mma_f16(acc[j][p], af[C::KS - 1], b.z, b.w);
                    } else {
#pragma unroll
                        for (int ks = 0; ks < C::KS; ++ks) {
                            const uint2 b = lds64(wa + ks * 8);
                            mma_f16(acc[j][p], af[ks], b.x, b.y);
                        }
                    }
                }

            // ---- the other terms, token by token
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = mt * 16 + h * 8 + tg;
                const int64_t tok = s * C::T + t;
                const uint32_t cfa = st + C::SC + t * C::CP;
                float v[4][4];
                const float4 qf = lds_f4(cfa + CF::kQ * 4);  // q, f
                const float f = qf.y * wdown;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[j][e] = acc[j][e >> 1][2 * h + (e & 1)] * f;
                if (a.g != nullptr) {
#pragma unroll
                    for (int k = 0; k < HC; ++k) {
                        const uint2 u = lds64(st + C::SG + t * C::GP + (k * C::CH + cl) * 2);
                        const float4 c = lds_f4(cfa + (k * HC + jq * 4) * 4);
                        const float gv[4] = {bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y)};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v[0][e] = fmaf(c.x, gv[e], v[0][e]);
                            v[1][e] = fmaf(c.y, gv[e], v[1][e]);
                            v[2][e] = fmaf(c.z, gv[e], v[2][e]);
                            v[3][e] = fmaf(c.w, gv[e], v[3][e]);
                        }
                    }
                }
                {
                    const uint2 u = lds64(st + C::SY + t * C::YP + cl * 2);
                    const float4 c = lds_f4(cfa + (CF::kPre + jq * 4) * 4);
                    const float yv[4] = {bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y)};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[0][e] = fmaf(c.x, yv[e], v[0][e]);
                        v[1][e] = fmaf(c.y, yv[e], v[1][e]);
                        v[2][e] = fmaf(c.z, yv[e], v[2][e]);
                        v[3][e] = fmaf(c.w, yv[e], v[3][e]);
                    }
                }
                // x, last: its operand is free once the products of step s - 1 are done
                if (K8 && h == 0) products_done();
                const bool in = tok < a.n && cl < width;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int jj = jq * 4 + j;
                    const uint32_t oa = (jj * (C::CH / 8) + grp * 2 + (tl >> 1)) * C::OT + t / 8 * 128 +
                                        t % 8 * 16 + (tl & 1) * 8;
                    float xv[4];
                    if (K8) {
                        const uint32_t c8 = lds32(st + C::SX + t * C::XP + jj * C::CH + cl);
                        const float sc = kept_scale(
                            smem[(s & 1) * C::STAGE + C::SS + (t * HC + jj) * (C::CH / 32) + cl / 32]);
                        e4m3x4_to_float(c8, xv);
#pragma unroll
                        for (int e = 0; e < 4; ++e) xv[e] *= sc;
                        sts64(sb + C::OO + oa, pack_bf16x2(xv[0], xv[1]), pack_bf16x2(xv[2], xv[3]));
                    } else {
                        const uint2 u = lds64(st + C::SX + oa);
                        xv[0] = bf16lo(u.x), xv[1] = bf16hi(u.x);
                        xv[2] = bf16lo(u.y), xv[3] = bf16hi(u.y);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[j][e] = fmaf(qf.x, xv[e], v[j][e]);
                    if (in)
                        __stcs(reinterpret_cast<uint2 *>(a.dx + tok * F + jj * a.d + ch0 + cl),
                               make_uint2(pack_bf16x2(v[j][0], v[j][1]),
                                          pack_bf16x2(v[j][2], v[j][3])));
                }
            }
            if (s + 1 < s1) keep_scale(s + 1, next_scale);
        }
        if (K8) {  // the last step's products
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before();
            __syncthreads();
            if (tid == 0) {
                tc_fence_after();
                issue(s1 - 1, s1 - 1 - s0);
            }
            ++commits;
        }
        products_done();
        tc_fence_after();

        // ---- this run's dW: lanes are features, columns the mix numbers
        float *out = a.dwp + (blockIdx.x + slice) * (int64_t)C::MIX * C::FT;
        for (int m = warp >> 2; m < C::MTILES; m += C::WARPS / 4) {
            const uint32_t ta = tmem + m * CF::kN + ((uint32_t)(warp & 3) << 21);
            float *of = out + m * 128 + (warp & 3) * 32 + lane;
            float v[CF::kN];
#pragma unroll
            for (int q = 0; q < CF::kN / 16; ++q) tmem_ld16(ta + q * 16, v + q * 16);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < CF::kN; ++i) asm volatile("" : "+f"(v[i]));  // used after the wait
#pragma unroll
            for (int i = 0; i < C::MIX; ++i)
                of[(int64_t)i * C::FT] =
                    CF::kProducts == 1 ? v[i] + (v[(C::MIX + i) % CF::kN] + v[(2 * C::MIX + i) % CF::kN])
                                       : v[i];
        }
        tc_fence_before();
        __syncthreads();  // before W, the operands and the sums are written anew
        tc_fence_after();
        step += s1 - s0;
    }
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
}

template <int HC, bool K8>
cudaError_t launch(const PreBackward &p, const MainArgs &m, const DeviceInfo &di, cudaStream_t s) {
    using C = Cfg<HC, K8>;
    const cudaError_t e = cudaFuncSetAttribute(
        k_dx_dw<HC, K8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    Args a;
    a.split = m.split;
    a.n = p.n, a.d = p.d, a.nblk = kept_blocks(p.d);
    a.dy = p.dy, a.x = static_cast<const uint8_t *>(p.x.data), a.xs = p.x.scales, a.w = p.w;
    a.g = p.dstream, a.dx = p.dx, a.cf = m.cf, a.du16 = m.du16, a.du3 = m.du3, a.dwp = m.dwp;
    a.err = di.err_word;
    return launch_overlapped(k_dx_dw<HC, K8>, dim3((unsigned)m.split.blocks), dim3(C::THREADS),
                             (size_t)C::SMEM, s, a);
}

}  // namespace

cudaError_t launch_dx_dw(const PreBackward &p, const MainArgs &m, const DeviceInfo &di,
                         cudaStream_t s) {
    const bool k8 = p.x.scales != nullptr;
    if (p.hc == 4) return k8 ? launch<4, true>(p, m, di, s) : launch<4, false>(p, m, di, s);
    return k8 ? launch<8, true>(p, m, di, s) : launch<8, false>(p, m, di, s);
}

}  // namespace hc
