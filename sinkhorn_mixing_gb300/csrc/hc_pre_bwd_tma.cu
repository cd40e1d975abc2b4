// hc_pre_bwd_tma.cu -- dx and dW of hc_mixes_pre's gradient at hc = 4, streamed
// by TMA (hc_pre_bwd.cu has the formulas; hc_pre_bwd_main.cu does the other
// shapes).
//
// A block owns 64 channels of all four copies (256 features) and walks over
// tokens in steps of 32 (Split).  Both products run on tcgen05:
//   du W    [32 tokens, 256 features], K = 24: one product a step into TMEM,
//     fp16 operands times powers of two (as in hc_pre_bwd_main.cu).  The 32
//     tokens stand in the 128 rows four times, so that every warp finds them in
//     the lanes it can read.
//   du^T x  [256 features, 24], K = tokens: sums over the steps in TMEM, x as
//     kept in bf16 (codes are widened into an operand tile on the way), du in
//     three bf16 parts.
// The rest is per token and channel: a lane is one token, and its coefficients
// serve 8 channels of 4 copies.  dx leaves by a TMA store, from the stage's
// gradient tile; of codes, that tile takes the widened x instead and dx has a
// tile of its own, so that the stage is free once the products are done.
// Roles: warps 0-7 compute the even steps and warps 8-15 the odd ones, so that
// one group's arithmetic runs under the other's waits; warp 16 loads (one
// thread), warp 17 issues the products, warp 18 stores.  Four stages; every wait
// has a limit, and after one ran out all roles run through without acting, so
// that all barriers are met.
// 16,384 tokens of 4 x 5120 in 8 bits (1.86 GB): 376 us, 4.9 TB/s; 65,536: 1,440 us, 5.2 TB/s.
// (With steps of 64 tokens, two stages and all 16 warps on each step 65,536 tokens
// of 4 x 5120 in 8 bits took 1,994 us in all, this way 1,828.)
#include <cuda_fp16.h>

#include "hc_loads.h"
#include "hc_pre_bwd.cuh"
#include "hc_pre_bwd.h"

namespace hc {
namespace {

using namespace ptx;
using CF = Coef<4>;

constexpr int T = kTileTokens, CH = 64, FT = 4 * CH, MIX = 24;
constexpr int kGroupWarps = 8, kComputeWarps = 2 * kGroupWarps;
constexpr int kThreads = 32 * (kComputeWarps + 3);
constexpr int kStages = 4;
// Steps between moves of dW's running sums (32 products each).  Even: the moves of a run are
// all one group's.
constexpr int kDrain = 16;

template <bool K8>
struct Lay {
    static constexpr int X = T * FT * (K8 ? 1 : 2), OX = T * FT * 2, OY = OX + X;
    static constexpr int OR = OY + T * CH * 2;
    static constexpr int STAGE = OR + CF::kTileBytes;
    static constexpr int OO = kStages * STAGE;                 // dx on its way out (K8)
    static constexpr int OW = OO + (K8 ? T * FT * 2 : 0);      // W, 32 halves a feature
    static constexpr int OS = OW + FT * 64;                    // scales [group][2][2 blocks][T][4]
    static constexpr int OE = OS + (K8 ? 2 * 2 * 2 * T * 16 : 0);  // barriers, flags, maxima
    static constexpr int SMEM = OE + 512;
    static_assert(STAGE % 1024 == 0 && OW % 1024 == 0, "swizzled tiles");
    static_assert(SMEM <= 232448, "shared memory");
};

// Barriers: one a stage, and below those one for even and one for odd steps, as a wait
// names a phase by its parity and each group sees every second step.
enum Bar { kFull = 0, kEmpty = 32, kOut = 64, kD1Full = 96, kD1Free = 112, kGate = 128,
           kD2Done = 144, kOutFree = 160 };
constexpr int kAbort = 176, kTmem = 180, kLast = 184, kMaxima = 192;
constexpr int kD2 = 256, kSums = kD2 + 2 * CF::kN;  // TMEM columns; du W has 0..255
static_assert(kSums + 2 * MIX <= 512, "TMEM");

constexpr uint32_t kIdescW = (1u << 4) | ((uint32_t)(FT >> 3) << 17) | (8u << 24);  // fp16
constexpr uint32_t kIdescX = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                             ((uint32_t)(CF::kN >> 3) << 17) | (8u << 24);          // bf16

struct Args {
    Split split;
    int64_t n, d;
    const uint8_t *xs;  // [steps][slices][T][4 copies][2 blocks], one slice's of a step together
    const float *w;
    const uint8_t *rec;
    float *dwp;
    unsigned int *err;
    int has_g;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1,
                                            int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, int c0, int c1, int c2,
                                             uint32_t src) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(c0), "r"(c1), "r"(c2), "r"(src)
        : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const uint8_t *src, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
// Has the barrier's phase of this parity ended?  Does not wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
template <int ID, int N>
__device__ __forceinline__ void meet() {
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(N) : "memory");
}

// Matrix descriptor of rows of 128 bytes (64 features) with 128-byte swizzle, rows
// along K; T tokens to the next 64 features.
__device__ __forceinline__ uint64_t tiles128(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(T * 128 >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Walks the runs of steps of this block: f(slice, partial sums, first step,
// past the last).
template <typename Fn>
__device__ __forceinline__ void over_runs(const Split &sp, Fn f) {
    const int64_t team = blockIdx.x / sp.wide, place = blockIdx.x % sp.wide;
    int64_t step = sp.first(team);
    const int64_t end = sp.first(team + 1);
    while (step < end) {
        const int64_t band = step / sp.steps, s0 = step - band * sp.steps;
        const int64_t s1 = min(sp.steps, s0 + (end - step));
        f(band * sp.wide + place, (team + band) * sp.wide + place, s0, s1);
        step += s1 - s0;
    }
}

template <bool K8>
__global__ void __launch_bounds__(kThreads, 1)
    k_dx_dw_tma(const __grid_constant__ CUtensorMap map_g, const __grid_constant__ CUtensorMap map_x,
                const __grid_constant__ CUtensorMap map_y,
                const __grid_constant__ CUtensorMap map_dx, Args a) {
    using L = Lay<K8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = su32(smem), eb = sb + L::OE;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort = reinterpret_cast<int *>(smem + L::OE + kAbort);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::OE + kTmem);
    float *maxima = reinterpret_cast<float *>(smem + L::OE + kMaxima);  // per warp

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(eb + kFull + 8 * i, 1);
            mbar_init(eb + kEmpty + 8 * i, K8 ? 1 : 2);  // products; and the store
            mbar_init(eb + kOut + 8 * i, kGroupWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(eb + kD1Full + 8 * i, 1);
            mbar_init(eb + kD1Free + 8 * i, kGroupWarps);
            mbar_init(eb + kGate + 8 * i, kGroupWarps);
            mbar_init(eb + kD2Done + 8 * i, 1);
            mbar_init(eb + kOutFree + 8 * i, 1);
        }
        mbar_init(eb + kLast, 1);
        *abort = 0;
        if ((sb & 1023u) != 0) {  // swizzled tiles need it
            atomicOr(a.err, kErrSmemLayout);
            *abort = 1;
        }
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
    for (int q = tid; q < FT * 64 / 16; q += kThreads)  // W's rows behind the mix numbers: zeros
        sts128(sb + L::OW + q * 16, make_uint4(0, 0, 0, 0));
    __syncthreads();
    // wait_bar reads the timer, which takes long, so the waits of a healthy run end before it
    auto wait = [&](uint32_t bar, uint32_t parity) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try(eb + bar, parity & 1)) return true;
        return wait_bar<false>(eb + bar, parity & 1, abort, a.err);
    };
    // step i's barrier of a stage (its use i / kStages), and of its parity (i / 2)
    auto at_stage = [](Bar b, int64_t i) { return (uint32_t)b + (uint32_t)(i % kStages) * 8; };
    auto at_parity = [](Bar b, int64_t i) { return (uint32_t)b + (uint32_t)(i & 1) * 8; };
    auto wait_stage = [&](Bar b, int64_t i) {
        return wait(at_stage(b, i), (uint32_t)(i / kStages));
    };
    auto wait_parity = [&](Bar b, int64_t i) { return wait(at_parity(b, i), (uint32_t)(i >> 1)); };
    auto stage = [&](int64_t i) { return sb + (uint32_t)(i % kStages) * L::STAGE; };
    int64_t it = 0;  // steps of this block so far

    if (warp == kComputeWarps) {
        // ------------------------------------------------------- loads
        if (lane == 0) {
            griddep_wait_then_release();
            asm volatile("fence.proxy.async;" ::: "memory");  // records were plain stores
            RingLoads<kStages> loads;
            over_runs(a.split, [&](int64_t slice, int64_t, int64_t s0, int64_t s1) {
                for (int64_t s = s0; s < s1; ++s, ++it) {
                    if (it >= kStages && !wait_stage(kEmpty, it - kStages)) continue;
                    if (*abort) continue;
                    loads.issue();
                    const uint32_t st = stage(it), bar = eb + at_stage(kFull, it);
                    mbar_expect_tx(bar, L::X + T * CH * 2 + CF::kTileBytes +
                                            (a.has_g ? T * FT * 2 : 0));
                    const int c = (int)slice * CH, t = (int)(s * T);
                    if (a.has_g) tma_load_3d(st, &map_g, c, t, 0, bar);
                    tma_load_3d(st + L::OX, &map_x, c, t, 0, bar);
                    bulk_load(st + L::OR, a.rec + s * CF::kTileBytes, CF::kTileBytes, bar);
                    tma_load_2d(st + L::OY, &map_y, c, t, bar);
                }
            });
            // what was loaded has to land before this block ends, waited for by others or not
            loads.in_flight([&](int stage, uint32_t parity) {
                settle_bar(eb + kFull + 8 * stage, parity);
            });
        }
    } else if (warp == kComputeWarps + 1) {
        // ---------------------------------------------------- products
        over_runs(a.split, [&](int64_t, int64_t, int64_t s0, int64_t s1) {
            meet<2, 32 * (kComputeWarps + 1)>();  // W of this slice is there
            if (lane == 0) {
                // Both products of a step as soon as each can go: du^T x must not wait for the
                // next step's tiles (its stage would not be loaded meanwhile), nor du W of the
                // next step for this one's operand.
                const int64_t i0 = it, end = it + (s1 - s0);
                int64_t next = it;  // step of du W; `it` that of du^T x
                uint64_t since = 0;  // the timer at the first of many idle rounds
                uint32_t rounds = 0;
                while (it < end) {
                    bool idle = true;
                    if (next < end &&
                        mbar_test(eb + at_stage(kFull, next), (uint32_t)(next / kStages) & 1) &&
                        (next == 0 || mbar_test(eb + at_parity(kD1Free, next - 1),
                                                (uint32_t)((next - 1) >> 1) & 1))) {
                        tc_fence_after();
                        const uint32_t ao = stage(next) + L::OR + T * CF::kTileCoefBytes;
#pragma unroll
                        for (int ks = 0; ks < CF::kK / 16; ++ks)
                            mma_bf16(tmem, rows16(ao + ks * 256, 128, 512),
                                     rows16(sb + L::OW + ks * 256, 128, 512), kIdescW, ks > 0);
                        mma_commit(eb + at_parity(kD1Full, next));
                        ++next;
                        idle = false;
                    }
                    if (it < next &&
                        mbar_test(eb + at_parity(kGate, it), (uint32_t)(it >> 1) & 1)) {
                        tc_fence_after();
                        const uint32_t xo = stage(it) + (K8 ? 0 : L::OX);
                        const uint32_t bo =
                            stage(it) + L::OR + T * CF::kTileCoefBytes + 128 * CF::kKBytes;
#pragma unroll
                        for (int ks = 0; ks < T / 16; ++ks)
#pragma unroll
                            for (int m = 0; m < 2; ++m)
                                mma_bf16(tmem + kD2 + m * CF::kN,
                                         tiles128(xo + m * 2 * T * 128 + ks * 2048),
                                         rows16(bo + ks * 256, 128, T / 8 * 128), kIdescX,
                                         (it - i0) % kDrain != 0 || ks > 0);
                        mma_commit(eb + at_parity(kD2Done, it));
                        mma_commit(eb + at_stage(kEmpty, it));
                        ++it;
                        idle = false;
                    }
                    rounds = idle ? rounds + 1 : 0;
                    if (idle) __nanosleep(40);  // the scheduler's other warps compute
                    if (rounds != 0 && rounds % 4096 == 0) {
                        if (*abort) break;
                        if (rounds == 4096) since = gtimer();
                        if (gtimer() - since > kTimeoutNs) {
                            *abort = 1;
                            atomicOr(a.err, kErrWaitTimeout);
                        }
                    }
                }
                it = end;
            }
            __syncwarp();
        });
        if (lane == 0) settle_products(eb + kLast);
    } else if (warp == kComputeWarps + 2) {
        // ------------------------------------------------------ stores
        if (lane == 0) {
            over_runs(a.split, [&](int64_t slice, int64_t, int64_t s0, int64_t s1) {
                for (int64_t s = s0; s < s1; ++s, ++it) {
                    if (!wait_stage(kOut, it) || *abort) continue;
                    if (slice * CH < a.d)  // else behind the last channel (Split)
                        tma_store_3d(&map_dx, (int)slice * CH, (int)(s * T), 0,
                                     K8 ? sb + L::OO : stage(it));
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    mbar_arrive(eb + (K8 ? at_parity(kOutFree, it) : at_stage(kEmpty, it)));
                }
            });
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
    } else {
        // ----------------------------------------------------- compute
        // lane's token of the step is `lane`; the warp's group and 8 channels
        const int group = warp / kGroupWarps, tl = lane, cg = (warp >> 2 & 1) * 4 + (warp & 3);
        const int gt = tid % (32 * kGroupWarps);
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        const uint32_t row = (uint32_t)tl * 128 + (uint32_t)((cg ^ (tl & 7)) << 4);
        const uint32_t row8 =
            (uint32_t)tl * 64 + (uint32_t)(((cg >> 1) ^ (tl >> 1 & 3)) << 4) + (cg & 1) * 8;
        const int64_t F = 4 * a.d;
        auto arrive = [&](uint32_t bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive(eb + bar);
        };
        bool started = false;
        over_runs(a.split, [&](int64_t slice, int64_t partial, int64_t s0, int64_t s1) {
            const int64_t ch0 = slice * CH;
            const int width = (int)min((int64_t)CH, a.d - ch0);
            // ---- the slice of W in fp16, its largest magnitude brought to [2^13, 2^14): 8 x 8
            // blocks [feature group][mix group][feature][mix]
            constexpr int kW = MIX * FT / 4 / (32 * kComputeWarps);
            float top = 0.0f;
            float4 wv[kW];  // all of it in flight at once
#pragma unroll
            for (int r = 0; r < kW; ++r) {
                const int q = (r * 32 * kComputeWarps + tid) * 4, i = q / FT, f = q % FT;
                wv[r] = f % CH < width
                            ? __ldg(reinterpret_cast<const float4 *>(
                                  a.w + (int64_t)i * F + f / CH * a.d + ch0 + f % CH))
                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                top = fmaxf(fmaxf(fmaxf(fabsf(wv[r].x), fabsf(wv[r].y)),
                                  fmaxf(fabsf(wv[r].z), fabsf(wv[r].w))),
                            top);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
            if (lane == 0) maxima[warp] = top;
            meet<1, 32 * kComputeWarps>();
            top = maxima[lane % kComputeWarps];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
            const int ex = min(max((int)(__float_as_uint(top) >> 23), 14), 253);
            const float wup = __uint_as_float((uint32_t)(267 - ex) << 23);
            const float wdown = __uint_as_float((uint32_t)(ex - 13) << 23);
#pragma unroll
            for (int r = 0; r < kW; ++r) {
                const int q = (r * 32 * kComputeWarps + tid) * 4, i = q / FT, f = q % FT;
                const float w4[4] = {wv[r].x, wv[r].y, wv[r].z, wv[r].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<__half *>(smem + L::OW + (f + e) / 8 * 512 + i / 8 * 128 +
                                                (f + e) % 8 * 16 + i % 8 * 2) =
                        __float2half_rn(w4[e] * wup);
            }
            if (!started) {
                griddep_wait_then_release();
                started = true;
            }

            // ---- this group's steps of the run
            const int64_t run = it, end = it + (s1 - s0);
            const int64_t own = run + ((run ^ group) & 1);
            // Scales: one a thread, loaded two of the group's steps ahead and passed on one ahead
            // through [block][token][copy].  Every warp reads a step's scales before it arrives
            // at that step's kD1Free and writes the next one's behind its own read, so a phase
            // of that barrier says both that they are there and that the other half is free.
            const int sct = gt >> 3, scj = gt >> 1 & 3, scb = gt & 1;
            const int64_t slices = (a.d + CH - 1) / CH;
            const uint8_t *sp = a.xs + ((s0 + (own - run)) * slices + slice) * (T * 8) + gt;
            auto load_scale = [&](int64_t i) -> uint32_t {
                uint32_t v = 0;
                if (K8 && i < end && slice < slices && (s0 + (i - run)) * T + sct < a.n)
                    v = __ldg(sp);
                sp += 2 * slices * (T * 8);
                return v;
            };
            const uint32_t sbuf = L::OS + group * (2 * 2 * T * 16);
            auto keep_scale = [&](int64_t i, uint32_t v) {
                if (K8)
                    *reinterpret_cast<float *>(smem + sbuf + (i >> 1 & 1) * (2 * T * 16) +
                                               (scb * T + sct) * 16 + scj * 4) = kept_scale(v);
            };
            // dW's sums so far move on (see hc_pre_bwd_main.cu); `out`: the run's result.  A
            // group's warps read 32 lanes of one of the two tiles each.
            auto drain = [&](bool first, float *out) {
                const int m = warp >> 2 & 1;
                const uint32_t ta = lanes + kD2 + m * CF::kN, ts = lanes + kSums + m * MIX;
#pragma unroll 1
                for (int c = 0; c < MIX; c += 8) {
                    float v[8], u[8], w[8], sum[8];
                    tmem_ld8(ta + c, v);
                    tmem_ld8(ta + MIX + c, u);
                    tmem_ld8(ta + 2 * MIX + c, w);
                    if (!first) tmem_ld8(ts + c, sum);
                    tmem_ld_wait();
                    arrived<8>(v);
                    arrived<8>(u);
                    arrived<8>(w);
                    if (!first) arrived<8>(sum);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] += u[e] + w[e];
                        if (!first) v[e] += sum[e];
                    }
                    if (out != nullptr) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            out[(int64_t)(c + e) * FT + m * 128 + (warp & 3) * 32 + lane] = v[e];
                    } else {
                        tmem_st8(ts + c, v);
                    }
                }
                tmem_st_wait();
            };

            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            keep_scale(own, load_scale(own));
            uint32_t next_scale = load_scale(own + 2);
            meet<2, 32 * (kComputeWarps + 1)>();
            for (int64_t i = own; i < end; i += 2) {
                const uint32_t st = stage(i);
                wait_stage(kFull, i);
                wait_parity(kD1Full, i);
                tc_fence_after();
                float4 sc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (K8) {
                    if (i >= 2) wait_parity(kD1Free, i - 2);
                    const uint4 u = lds128(sb + sbuf + (uint32_t)(i >> 1 & 1) * (2 * T * 16) +
                                           ((cg >> 2) * T + tl) * 16);
                    sc = make_float4(__uint_as_float(u.x), __uint_as_float(u.y),
                                     __uint_as_float(u.z), __uint_as_float(u.w));
                    keep_scale(i + 2, next_scale);
                    next_scale = load_scale(i + 4);
                }
                // ---- du W of this token
                uint64_t v[4][4], qq, ff;
                const uint32_t cfa = st + L::OR + tl * CF::kTileCoefBytes;
                {
                    float acc[4][8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) tmem_ld8(lanes + j * CH + cg * 8, acc[j]);
                    const uint2 u = lds64(cfa + CF::kQ * 4);
                    const float q = __uint_as_float(u.x), f = __uint_as_float(u.y) * wdown;
                    qq = pack2(q, q), ff = pack2(f, f);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 4; ++j) arrived<8>(acc[j]);
                    tc_fence_before();
                    arrive(at_parity(kD1Free, i));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int p = 0; p < 4; ++p)
                            v[j][p] = fmul2(pack2(acc[j][2 * p], acc[j][2 * p + 1]), ff);
                }
                // ---- the stream's gradient through comb, and y's through pre
                auto add = [&](uint32_t coef, const uint4 &u) {
                    const uint4 w = lds128(coef);
                    const uint64_t c[4] = {twice(w.x), twice(w.y), twice(w.z), twice(w.w)};
                    const uint64_t b[4] = {bf16x2_to_f32x2(u.x), bf16x2_to_f32x2(u.y),
                                           bf16x2_to_f32x2(u.z), bf16x2_to_f32x2(u.w)};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int p = 0; p < 4; ++p) ffma2(v[j][p], c[j], b[p]);
                };
                if (a.has_g) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) add(cfa + k * 16, lds128(st + k * T * 128 + row));
                }
                add(cfa + CF::kPre * 4, lds128(st + L::OY + row));
                // ---- x; widened codes go over the gradient's tile, which this lane has read
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint64_t xv[4];
                    if (K8) {
                        const float f1 = j == 0 ? sc.x : j == 1 ? sc.y : j == 2 ? sc.z : sc.w;
                        const uint64_t f2 = pack2(f1, f1);
                        float f[8];
                        e4m3x8_to_float(lds64(st + L::OX + j * T * 64 + row8), f);
#pragma unroll
                        for (int p = 0; p < 4; ++p)
                            xv[p] = fmul2(pack2(f[2 * p], f[2 * p + 1]), f2);
                        sts128(st + j * T * 128 + row,
                               make_uint4(pack_pair(xv[0]), pack_pair(xv[1]), pack_pair(xv[2]),
                                          pack_pair(xv[3])));
                    } else {
                        const uint4 u = lds128(st + L::OX + j * T * 128 + row);
                        xv[0] = bf16x2_to_f32x2(u.x), xv[1] = bf16x2_to_f32x2(u.y);
                        xv[2] = bf16x2_to_f32x2(u.z), xv[3] = bf16x2_to_f32x2(u.w);
                    }
#pragma unroll
                    for (int p = 0; p < 4; ++p) ffma2(v[j][p], qq, xv[p]);
                }
                // ---- du^T x may go, once the step before is through it (the other group's, which
                // is half a step ahead) and its sums have moved on where it is time
                if (K8) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                if (i > 0) wait_parity(kD2Done, i - 1);
                if (i > run && (i - run) % kDrain == 0) {
                    tc_fence_after();
                    drain(i - run == kDrain, nullptr);
                    tc_fence_before();
                }
                arrive(at_parity(kGate, i));
                if (K8 && i > 0) wait_parity(kOutFree, i - 1);
                const uint32_t out = K8 ? sb + L::OO : st;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sts128(out + j * T * 128 + row,
                           make_uint4(pack_pair(v[j][0]), pack_pair(v[j][1]), pack_pair(v[j][2]),
                                      pack_pair(v[j][3])));
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                arrive(at_stage(kOut, i));
            }
            it = end;
            if ((run & 1) == group) {
                wait_parity(kD2Done, end - 1);
                tc_fence_after();
                drain(s1 - s0 <= kDrain, a.dwp + partial * MIX * FT);
                tc_fence_before();
            }
            meet<1, 32 * kComputeWarps>();  // before maxima and W are written anew
        });
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
}

// [hc][n][d] view of a stream: boxes of 64 channels, T tokens, all copies.
bool stream_map(CUtensorMap *map, const void *p, bool bytes, int64_t n, int64_t d) {
    const cuuint64_t es = bytes ? 1 : 2;
    const cuuint64_t dim[3] = {(cuuint64_t)d, (cuuint64_t)n, 4};
    const cuuint64_t stride[2] = {(cuuint64_t)(4 * d) * es, (cuuint64_t)d * es};
    const cuuint32_t box[3] = {CH, T, 4}, one[3] = {1, 1, 1};
    return tensor_map_encoder()(
               map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<void *>(p), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               bytes ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               // more than a row of the box: what lies behind is read by the team's next block
               bytes ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool K8>
cudaError_t launch(const PreBackward &p, const MainArgs &m, const DeviceInfo &di, cudaStream_t s) {
    using L = Lay<K8>;
    static SmemState state;
    const cudaError_t e =
        allow_smem(state, reinterpret_cast<const void *>(k_dx_dw_tma<K8>), L::SMEM, di);
    if (e != cudaSuccess) return e;
    CUtensorMap g, x, y, dx;
    const cuuint64_t dim[2] = {(cuuint64_t)p.d, (cuuint64_t)p.n};
    const cuuint64_t stride[1] = {(cuuint64_t)p.d * 2};
    const cuuint32_t box[2] = {CH, T}, one[2] = {1, 1};
    if (!stream_map(&dx, p.dx, false, p.n, p.d) || !stream_map(&x, p.x.data, K8, p.n, p.d) ||
        !stream_map(&g, p.dstream != nullptr ? p.dstream : p.dx, false, p.n, p.d) ||
        tensor_map_encoder()(&y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                             const_cast<uint16_t *>(p.dy), dim, stride, box, one,
                             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    Args a;
    a.split = m.split;
    a.n = p.n, a.d = p.d;
    a.xs = m.scales, a.w = p.w, a.rec = m.rec, a.dwp = m.dwp, a.err = di.err_word;
    a.has_g = p.dstream != nullptr;
    return launch_overlapped(k_dx_dw_tma<K8>, dim3((unsigned)m.split.blocks()), dim3(kThreads),
                             (size_t)L::SMEM, s, g, x, y, dx, a);
}

}  // namespace

Split split_dx_dw_tma(int64_t n, int64_t d, int64_t most) { return Split::of(n, d, CH, T, most); }

// Four steps of tokens at least: below, the other kernel is as fast (8 tokens of
// 4 x 64: both are done before the host is) and needs no tensor maps.
bool dx_dw_tma_takes(const PreBackward &p) {
    return p.hc == 4 && p.d >= CH && p.n >= 4 * T && p.n < (int64_t(1) << 31) && forced_path() != kPathGeneral &&
           (p.x.scales == nullptr || p.d % 16 == 0) && tensor_map_encoder() != nullptr;
}

cudaError_t launch_dx_dw_tma(const PreBackward &p, const MainArgs &m, const DeviceInfo &di,
                             cudaStream_t s) {
    return p.x.scales != nullptr ? launch<true>(p, m, di, s) : launch<false>(p, m, di, s);
}

}  // namespace hc
