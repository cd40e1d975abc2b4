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
// step's loads running under this one's arithmetic.  4,096 tokens of 8 x 5120 in 8
// bits (0.9 GB): 412 us; no unit is full (LSU wavefronts 67%, issue slots 44%, DRAM 33%,
// tensor pipe 18%): all warps go through a step together, and nothing runs under its waits.
#include <cuda_fp16.h>
#include <type_traits>

#include "hc_pre_bwd.cuh"
#include "hc_pre_bwd.h"

namespace hc {
namespace {

using namespace ptx;

struct Args {
    Split split;
    int64_t n, d, nblk;
    const uint8_t *dy;      // bf16
    const uint8_t *x, *xs;  // bf16 rows or codes, scales
    const float *w;
    const uint8_t *g;       // bf16; may be null
    uint8_t *dx;            // bf16
    const uint8_t *rec;
    float *dwp;
    unsigned int *err;
};

constexpr int kDrain = 16;  // steps between moves of dW's running sums

template <int HC, bool K8>
struct Cfg {
    using CF = Coef<HC>;
    static constexpr int T = HC == 4 ? 32 : 16, CH = HC == 4 ? 128 : 64, FT = HC * CH;
    static constexpr int MIX = CF::kMix, KS = CF::kK / 16;
    // a warp: 16 tokens, 16 channels, NJ copies; a lane of it 2 tokens, 4 channels.  16 warps
    // (at hc = 8 with 4 copies there would be 8, and each step took twice as long)
    static constexpr int NJ = HC == 4 ? 4 : 2;
    static constexpr int MT = T / 16, GROUPS = CH / 16, JQ = HC / NJ, WARPS = MT * GROUPS * JQ;
    static constexpr int THREADS = 32 * WARPS, MTILES = FT / 128;
    static_assert(WARPS == 4 * MTILES, "a warp reads 32 lanes of one tile of dW");
    static constexpr int SUMS = MTILES * CF::kN;   // TMEM columns of the drained sums
    static constexpr int SUMT = (512 - SUMS) / CF::kMix;  // tiles that find room there
    // Row pitches: a token's row is moved on by as many bytes as the lanes of one token read at
    // once, so that the lanes of neighbouring tokens meet in no bank.
    static constexpr int GP = HC * CH * 2 + 32, YP = CH * 2 + 32, XP = HC * CH + 16;
    static constexpr int CP = CF::kCoefBytes, AP = CF::kKBytes + 16;
    // x as the M operand: 8 channels x 8 tokens in 128 bytes (channels along 16 bytes), the
    // blocks of a channel group's tokens in a row
    static constexpr int OT = T / 8 * 128, OBYTES = FT / 8 * OT;
    static constexpr int BT = T / 8 * 128, BBYTES = CF::kParts / 8 * BT;
    // stage
    static constexpr int SG = 0, SY = SG + T * GP, SX = SY + T * YP;
    static constexpr int SS = SX + (K8 ? T * XP : OBYTES);  // scales
    static constexpr int SCALES = T * HC * CH / 32;
    static constexpr int SC = SS + (K8 ? SCALES * 4 : 0), SA = SC + T * CP;
    static constexpr int STAGE = (SA + T * AP + 127) / 128 * 128;
    // the block's memory: two stages, a longer ring for du3, which products still under way read
    // (three stages, which would fit at HC = 8 in 8 bits, took longer: 4,096 tokens of 8 x 5120
    // 607 us against 525 for two in the same build)
    static constexpr int BRING = K8 ? 3 : 2;
    static constexpr int OB = 2 * STAGE, OO = OB + BRING * BBYTES;  // du3 ring; x operand (K8)
    static constexpr int OW = OO + (K8 ? OBYTES : 0), WREG = 2 * KS;
    static constexpr int WBYTES = FT / 8 * 32 * WREG * 4;
    static constexpr int WV = MIX * FT / 4 / THREADS;               // float4 of W a thread
    static_assert(WV * 4 * THREADS == MIX * FT, "W splits over the threads");
    static constexpr int OE = OW + WBYTES;                          // barrier, flags, maxima
    static constexpr int SMEM = OE + 256;
    static constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                                      ((uint32_t)(CF::kN >> 3) << 17) | (8u << 24);
    static_assert(WARPS % 2 == 0 && 16 + WARPS * 4 + 8 <= 256, "barriers, flags, maxima");
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(SCALES <= THREADS, "a scale byte per thread");
};

// Asynchronous copies of 16 (8) bytes of which `bytes` are read, zeros behind.
__device__ __forceinline__ void cp16(uint32_t dst, const uint8_t *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const uint8_t *src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_wait_all() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
// N floats, each twice
template <int N>
__device__ __forceinline__ void lds_twice(uint32_t a, uint64_t (&v)[N]) {
    if (N == 4) {
        const uint4 u = lds128(a);
        v[0] = twice(u.x), v[1] = twice(u.y), v[N - 2] = twice(u.z), v[N - 1] = twice(u.w);
    } else {
        const uint2 u = lds64(a);
        v[0] = twice(u.x), v[1] = twice(u.y);
    }
}
// c = a b (first) or c += a b
template <bool FIRST>
__device__ __forceinline__ void mma_f16(float c[4], const uint32_t a[4], uint32_t b0,
                                        uint32_t b1) {
    if (FIRST)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// a streaming store where `in` is not 0, without a branch around it
__device__ __forceinline__ void stg64_if(uint8_t *p, uint32_t x, uint32_t y, uint32_t in) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t@p st.global.cs.v2.u32 [%0], {%1, %2};\n\t}" ::"l"(
            p),
        "r"(x), "r"(y), "r"(in)
        : "memory");
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
    const uint32_t last = sb + C::OE + 16 + C::WARPS * 4;  // barrier of the end, after a timeout

    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(last, 1);
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
    if (CF::kK > C::MIX)  // the rows of W behind the mix numbers stay zero
        for (int q = tid; q < C::WBYTES / 16; q += C::THREADS)
            sts128(sb + C::OW + q * 16, make_uint4(0, 0, 0, 0));
    __syncthreads();

    // lane's place: tokens mt*16 + lane/4 (+ 8), channels cl .. cl+3 of the slice, copies jq*4 ..
    const int mt = warp % C::MT, grp = warp / C::MT % C::GROUPS, jq = warp / (C::MT * C::GROUPS);
    const int tg = lane >> 2, tl = lane & 3, cl = grp * 16 + tl * 4;
    const int64_t F = HC * a.d;
    uint32_t commits = 0;  // products committed to `bar` so far
    auto products_done = [&] {
        return commits == 0 || wait_bar<false>(bar, (commits - 1) & 1, abort, a.err);
    };

    bool started = false;  // has this kernel waited for the one before it
    const int64_t team = blockIdx.x / a.split.wide, place = blockIdx.x % a.split.wide;
    int64_t step = a.split.first(team);
    const int64_t end = a.split.first(team + 1);
    while (step < end) {
        const int64_t band = step / a.split.steps;
        const int64_t s0 = step - band * a.split.steps;
        const int64_t s1 = min(a.split.steps, s0 + (end - step));
        // (a band's last slices may lie behind the last channel: nothing there is read or kept)
        const int64_t slice = band * a.split.wide + place;
        const int64_t ch0 = slice * C::CH < a.d ? slice * C::CH : 0;
        const int width = (int)max((int64_t)0, min((int64_t)C::CH, a.d - slice * C::CH));

        // ---- the slice of W, in fp16 times a power of two that brings its largest magnitude
        // to [2^13, 2^14), laid out as the products' B fragments
        float top = 0.0f;
        float4 wv[C::WV];  // all of it in flight at once
#pragma unroll
        for (int r = 0; r < C::WV; ++r) {
            const int q = (r * C::THREADS + tid) * 4, i = q / C::FT, f = q % C::FT;
            wv[r] = f % C::CH < width
                        ? __ldg(reinterpret_cast<const float4 *>(a.w + (int64_t)i * F +
                                                                 f / C::CH * a.d + ch0 + f % C::CH))
                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            top = fmaxf(fmaxf(fmaxf(fabsf(wv[r].x), fabsf(wv[r].y)),
                              fmaxf(fabsf(wv[r].z), fabsf(wv[r].w))),
                        top);
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
#pragma unroll
        for (int r = 0; r < C::WV; ++r) {
            const int q = (r * C::THREADS + tid) * 4, i = q / C::FT, f = q % C::FT;
            const float w4[4] = {wv[r].x, wv[r].y, wv[r].z, wv[r].w};
            const int k = i & 15, reg = (i >> 4) * 2 + (k >> 3);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // channel 4 t + 2 p + b of its group of 16 is row n = 2 t + b of product p
                const int c = f % C::CH + e, g = (c >> 2 & 3) * 2 + (e & 1), p = e >> 1;
                const int nt = (f / C::CH * C::GROUPS + (c >> 4)) * 2 + p, ln = g * 4 + (k & 7) / 2;
                reinterpret_cast<__half *>(
                    smem + C::OW)[((nt * 32 + ln) * C::WREG + reg) * 2 + (k & 1)] =
                    __float2half_rn(w4[e] * wup);
            }
        }
        if (!started) {
            griddep_wait_then_release();
            started = true;
        }

        // ---- loads of one step's tiles.  A thread's pieces of 16 bytes lie at one column of
        // every GT-th row (YT-th, XT-th), so a pointer per tensor walks over them, and the columns
        // past the slice's end read 0 bytes at column 0.
        constexpr int GT = C::THREADS / (C::FT / 8), YT = C::THREADS / (C::CH / 8);
        constexpr int XV = C::FT / 16, XT = C::THREADS / XV;
        constexpr int RV = CF::kBytes / 16, R1 = CF::kCoefBytes / 16, R2 = R1 + CF::kKBytes / 16;
        constexpr int RN = (C::T * RV + C::THREADS - 1) / C::THREADS;
        const int gt = tid / (C::FT / 8), gv = tid % (C::FT / 8);
        const int gk = gv / (C::CH / 8), gc = gv % (C::CH / 8) * 8;
        const int yt = tid / (C::CH / 8), yc = tid % (C::CH / 8) * 8;
        const int xt = tid / XV, xv0 = tid % XV, xk = xv0 / (C::CH / 16), xc = xv0 % (C::CH / 16) * 16;
        const uint32_t gsz = gc < width ? 16 : 0, ysz = yc < width ? 16 : 0;
        const bool wide = K8 && a.d % 16 == 0;  // 16 codes are 16-byte aligned
        const uint32_t xsz = !K8 ? gsz : wide ? (xc < width ? 16 : 0) : gsz / 2;
        const int64_t gstep = GT * F * 2;
        const int64_t gat = gt * F + (gsz ? gk * a.d + gc : 0) + ch0;
        const uint8_t *gp = a.g + (s0 * C::T * F + gat) * 2;
        const uint8_t *yp = a.dy + ((s0 * C::T + yt) * a.d + ch0 + (ysz ? yc : 0)) * 2;
        const int64_t xstep = wide ? XT * F : K8 ? GT * F : gstep;
        const uint8_t *xp = !K8    ? a.x + (s0 * C::T * F + gat) * 2
                            : wide ? a.x + (s0 * C::T + xt) * F + (xsz ? xk * a.d + xc : 0) + ch0
                                   : a.x + s0 * C::T * F + gat;
        const uint8_t *rp = a.rec + s0 * C::T * CF::kBytes + tid * 16;
        uint32_t rdst[RN];  // in the stage, or (from C::STAGE on) in the ring of du3
#pragma unroll
        for (int i = 0; i < RN; ++i) {
            const int q = i * C::THREADS + tid, t = q / RV, v = q % RV;
            rdst[i] = v < R1   ? C::SC + t * C::CP + v * 16
                      : v < R2 ? C::SA + t * C::AP + (v - R1) * 16
                               : C::STAGE + (v - R2) * C::BT + t / 8 * 128 + t % 8 * 16;
        }
        // `whole`: all C::T tokens exist, else the first `left`
        auto load_rows = [&](int64_t s, int64_t rel, auto whole, int left) {
            constexpr bool W = decltype(whole)::value;
            const uint32_t st = sb + (uint32_t)(rel & 1) * C::STAGE;
            const uint32_t bt =
                sb + C::OB + (uint32_t)(rel % C::BRING) * C::BBYTES - C::STAGE;
            if (a.g != nullptr) {
                const uint8_t *p = gp;
#pragma unroll
                for (int i = 0; i < C::T / GT; ++i, p += gstep) {
                    const bool in = W || gt + i * GT < left;
                    cp16(st + C::SG + (gt + i * GT) * C::GP + gv * 16, in ? p : a.g, in ? gsz : 0);
                }
            }
            {
                const uint8_t *p = xp;
                const int n = wide ? C::T / XT : C::T / GT;
#pragma unroll
                for (int i = 0; i < C::T / GT; ++i, p += xstep) {
                    if (i >= n) break;
                    const int t = wide ? xt + i * XT : gt + i * GT;
                    const bool in = W || t < left;
                    const uint8_t *src = in ? p : a.x;
                    const uint32_t sz = in ? xsz : 0;
                    if (!K8)
                        cp16(st + C::SX + gv * C::OT + t / 8 * 128 + t % 8 * 16, src, sz);
                    else if (wide)
                        cp16(st + C::SX + t * C::XP + xv0 * 16, src, sz);
                    else
                        cp8(st + C::SX + t * C::XP + gv * 8, src, sz);
                }
            }
            static_assert(YT >= C::T, "one piece of dy a thread");
            if (YT == C::T || yt < C::T) {
                const bool in = W || yt < left;
                cp16(st + C::SY + yt * C::YP + yc * 2, in ? yp : a.dy, in ? ysz : 0);
            }
#pragma unroll
            for (int i = 0; i < RN; ++i) {
                const int q = i * C::THREADS + tid;
                const bool in = W || q / RV < left;
                if (q < C::T * RV)
                    cp16(rdst[i] + (rdst[i] < C::STAGE ? st : bt),
                         in ? rp + i * C::THREADS * 16 : a.rec, in ? 16 : 0);
            }
            gp += C::T * F * 2, yp += C::T * a.d * 2, xp += C::T * F * (K8 ? 1 : 2);
            rp += C::T * CF::kBytes;
        };
        auto load = [&](int64_t s, int64_t rel) {  // steps in order
            const int64_t left = a.n - s * C::T;
            if (left >= C::T)
                load_rows(s, rel, std::true_type(), C::T);
            else
                load_rows(s, rel, std::false_type(), (int)left);
        };
        // the scale byte of (token, block, copy) = tid of the next step
        const int sct = tid / (HC * (C::CH / 32)), scb = tid / HC % (C::CH / 32), scj = tid % HC;
        const bool sin = K8 && sct < C::T && scb * 32 < width;
        const uint8_t *sp =
            a.xs + ((s0 * C::T + (sin ? sct : 0)) * HC + scj) * a.nblk + ch0 / 32 + (sin ? scb : 0);
        auto load_scale = [&](int64_t s) -> uint32_t {
            uint32_t v = 0;
            if (sin && s * C::T + sct < a.n) v = __ldg(sp);
            sp += C::T * HC * a.nblk;
            return v;
        };
        auto keep_scale = [&](int64_t rel, uint32_t v) {
            if (K8 && tid < C::SCALES)
                reinterpret_cast<float *>(smem + (rel & 1) * C::STAGE + C::SS)[tid] =
                    kept_scale(v);
        };
        // dW += du^T x of the step `rel` of this run: one thread issues
        auto issue = [&](int64_t rel) {
            const uint32_t xo =
                K8 ? sb + C::OO : sb + (uint32_t)(rel & 1) * C::STAGE + C::SX;
            const uint32_t bo = sb + C::OB + (uint32_t)(rel % C::BRING) * C::BBYTES;
#pragma unroll
            for (int ks = 0; ks < C::T / 16; ++ks)
#pragma unroll
                for (int m = 0; m < C::MTILES; ++m)
#pragma unroll
                    for (int p = 0; p < CF::kProducts; ++p)
                        mma_bf16(tmem + m * CF::kN,
                                 rows16(xo + m * 16 * C::OT + ks * 256, 128, C::OT),
                                 rows16(bo + p * (CF::kN / 8) * C::BT + ks * 256, 128, C::BT),
                                 C::IDESC, rel % kDrain != 0 || ks > 0 || p > 0);
            mma_commit(bar);
        };

        // The tensor core rounds its running sums toward zero, which over many steps adds up to
        // more than binary32's own rounding.  So every kDrain steps the sums move on: into TMEM
        // columns of their own or, where those are taken (two of the tiles at HC = 8), to the
        // place of the run's result, added there with rounding to nearest; the products then
        // start anew.
        float *const result = a.dwp + ((team + band) * a.split.wide + place) * C::MIX * C::FT;
        auto drain = [&](bool first, bool last) {
            const int m = warp >> 2;
            const bool inside = m < C::SUMT;
            const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
            const uint32_t ta = lanes + m * CF::kN, ts = lanes + C::SUMS + m * C::MIX;
            float *of = result + m * 128 + (warp & 3) * 32 + lane;
#pragma unroll 1
            for (int c = 0; c < C::MIX; c += 8, of += 8 * C::FT) {
                float v[8], u[8], w[8], sum[8];
                tmem_ld8(ta + c, v);
                if (CF::kProducts == 1) {
                    tmem_ld8(ta + C::MIX + c, u);
                    tmem_ld8(ta + 2 * C::MIX + c, w);
                }
                if (!first) {
                    if (inside) {
                        tmem_ld8(ts + c, sum);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum[e] = of[e * C::FT];
                    }
                }
                tmem_ld_wait();
                arrived<8>(v);
                if (CF::kProducts == 1) {
                    arrived<8>(u);
                    arrived<8>(w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += u[e] + w[e];
                }
                if (!first) {
                    arrived<8>(sum);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += sum[e];
                }
                if (last || !inside) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) of[e * C::FT] = v[e];
                } else {
                    tmem_st8(ts + c, v);
                }
            }
            tmem_st_wait();
        };

        uint8_t *dxp =
            a.dx + ((s0 * C::T + mt * 16 + tg) * F + jq * C::NJ * a.d + ch0 + (cl < width ? cl : 0)) * 2;
        load(s0, 0);
        keep_scale(0, load_scale(s0));
        for (int64_t s = s0; s < s1; ++s) {
            const int64_t rel = s - s0;
            const bool full = rel > 0 && rel % kDrain == 0;
            cp_wait_all();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before();
            __syncthreads();  // step s has landed; all are done with step s - 1
            if (!K8 && rel > 0) {
                products_done();  // of step s - 1, whose x is loaded over
                if (full) {
                    tc_fence_after();
                    drain(rel == kDrain, false);
                    tc_fence_before();
                    __syncthreads();
                }
            }
            if (tid == 0 && (!K8 || rel > 0)) {
                tc_fence_after();
                issue(K8 ? rel - 1 : rel);
            }
            if (!K8 || rel > 0) ++commits;
            // The next step's loads go into the stage that step s - 1 has left.  Two of each
            // scheduler's four warps issue theirs before du W and two behind it, so that the
            // loads and the products of a step run beside each other (4,096 tokens of 8 x 5120
            // in 8 bits 498 -> 487 us, in bf16 537 -> 532; all behind it 540).  The condition is
            // formed twice from `warp`: a register that held it would spill others (502).
            uint32_t next_scale = 0;
            if (s + 1 < s1 && (warp & 4)) load(s + 1, rel + 1), next_scale = load_scale(s + 1);

            // ---- du W
            const uint32_t st = sb + (uint32_t)(rel & 1) * C::STAGE;
            float acc[C::NJ][2][4];
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
            for (int j = 0; j < C::NJ; ++j)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint32_t wa =
                        sb + C::OW +
                        ((((jq * C::NJ + j) * C::GROUPS + grp) * 2 + p) * 32 + lane) * C::WREG * 4;
                    if (C::KS == 2) {
                        const uint4 b = lds128(wa);
                        mma_f16<true>(acc[j][p], af[0], b.x, b.y);
                        mma_f16<false>(acc[j][p], af[C::KS - 1], b.z, b.w);
                    } else {
#pragma unroll
                        for (int ks = 0; ks < C::KS; ++ks) {
                            const uint2 b = lds64(wa + ks * 8);
                            if (ks == 0)
                                mma_f16<true>(acc[j][p], af[ks], b.x, b.y);
                            else
                                mma_f16<false>(acc[j][p], af[ks], b.x, b.y);
                        }
                    }
                }

            if (s + 1 < s1 && !(warp & 4)) load(s + 1, rel + 1), next_scale = load_scale(s + 1);

            // ---- the other terms, token by token, two channels wide
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = mt * 16 + h * 8 + tg;
                const uint32_t cfa = st + C::SC + t * C::CP + jq * C::NJ * 4;
                uint64_t v[C::NJ][2], qq, ff;
                {
                    const uint2 u = lds64(st + C::SC + t * C::CP + CF::kQ * 4);
                    const float q = __uint_as_float(u.x), f = __uint_as_float(u.y) * wdown;
                    qq = pack2(q, q), ff = pack2(f, f);
                }
#pragma unroll
                for (int j = 0; j < C::NJ; ++j)
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        v[j][p] = fmul2(pack2(acc[j][p][2 * h], acc[j][p][2 * h + 1]), ff);
                auto add = [&](uint32_t coef, const uint2 &u) {  // v_j += coef_j u
                    uint64_t c[C::NJ];
                    lds_twice(coef, c);
                    const uint64_t lo = bf16x2_to_f32x2(u.x), hi = bf16x2_to_f32x2(u.y);
#pragma unroll
                    for (int j = 0; j < C::NJ; ++j) {
                        ffma2(v[j][0], c[j], lo);
                        ffma2(v[j][1], c[j], hi);
                    }
                };
                if (a.g != nullptr) {
#pragma unroll
                    for (int k = 0; k < HC; ++k)
                        add(cfa + k * HC * 4, lds64(st + C::SG + t * C::GP + (k * C::CH + cl) * 2));
                }
                add(cfa + CF::kPre * 4, lds64(st + C::SY + t * C::YP + cl * 2));
                // x, last: its operand is free once the products of step s - 1 are done
                if (K8 && h == 0) products_done();
                const uint32_t in = cl < width && (s * C::T + t < a.n);
                uint8_t *p = dxp + h * 16 * F;
                uint64_t sc[C::NJ];
                if (K8) {
                    lds_twice(st + C::SS + ((t * (C::CH / 32) + cl / 32) * HC + jq * C::NJ) * 4, sc);
                }
#pragma unroll
                for (int j = 0; j < C::NJ; ++j, p += a.d * 2) {
                    const int jj = jq * C::NJ + j;
                    const uint32_t oa = (jj * (C::CH / 8) + grp * 2 + (tl >> 1)) * C::OT + t / 8 * 128 +
                                        t % 8 * 16 + (tl & 1) * 8;
                    uint64_t xv[2];
                    if (K8) {
                        float f[4];
                        e4m3x4_to_float(lds32(st + C::SX + t * C::XP + jj * C::CH + cl), f);
                        xv[0] = fmul2(pack2(f[0], f[1]), sc[j]);
                        xv[1] = fmul2(pack2(f[2], f[3]), sc[j]);
                        sts64(sb + C::OO + oa, pack_pair(xv[0]), pack_pair(xv[1]));
                    } else {
                        const uint2 u = lds64(st + C::SX + oa);
                        xv[0] = bf16x2_to_f32x2(u.x), xv[1] = bf16x2_to_f32x2(u.y);
                    }
                    ffma2(v[j][0], qq, xv[0]);
                    ffma2(v[j][1], qq, xv[1]);
                    stg64_if(p, pack_pair(v[j][0]), pack_pair(v[j][1]), in);
                }
            }
            dxp += C::T * F * 2;
            if (s + 1 < s1) keep_scale(rel + 1, next_scale);
            if (K8 && full) {  // the products up to step s - 1 are done
                tc_fence_after();
                drain(rel == kDrain, false);
            }
        }
        if (K8) {  // the last step's products
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before();
            __syncthreads();
            if (tid == 0) {
                tc_fence_after();
                issue(s1 - 1 - s0);
            }
            ++commits;
        }
        products_done();
        tc_fence_after();
        drain(s1 - s0 <= kDrain, true);
        tc_fence_before();
        __syncthreads();  // before W, the operands and the sums are written anew
        tc_fence_after();
        step += s1 - s0;
    }
    if (tid == 0 && *abort) settle_products(last);  // what a wait gave up on
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
}

template <int HC, bool K8>
cudaError_t launch(const PreBackward &p, const MainArgs &m, const DeviceInfo &di, cudaStream_t s) {
    using C = Cfg<HC, K8>;
    static SmemState state;
    const cudaError_t e =
        allow_smem(state, reinterpret_cast<const void *>(k_dx_dw<HC, K8>), C::SMEM, di);
    if (e != cudaSuccess) return e;
    Args a;
    a.split = m.split;
    a.n = p.n, a.d = p.d, a.nblk = kept_blocks(p.d);
    a.dy = reinterpret_cast<const uint8_t *>(p.dy), a.x = static_cast<const uint8_t *>(p.x.data), a.xs = p.x.scales, a.w = p.w;
    a.g = reinterpret_cast<const uint8_t *>(p.dstream);
    a.dx = reinterpret_cast<uint8_t *>(p.dx), a.rec = m.rec, a.dwp = m.dwp;
    a.err = di.err_word;
    return launch_overlapped(k_dx_dw<HC, K8>, dim3((unsigned)m.split.blocks()), dim3(C::THREADS),
                             (size_t)C::SMEM, s, a);
}

}  // namespace

Split split_dx_dw(int64_t n, int hc, int64_t d, int64_t most) {
    return hc == 4 ? Split::of(n, d, Cfg<4, true>::CH, Cfg<4, true>::T, most)
                   : Split::of(n, d, Cfg<8, true>::CH, Cfg<8, true>::T, most);
}

cudaError_t launch_dx_dw(const PreBackward &p, const MainArgs &m, const DeviceInfo &di,
                         cudaStream_t s) {
    const bool k8 = p.x.scales != nullptr;
    if (p.hc == 4) return k8 ? launch<4, true>(p, m, di, s) : launch<4, false>(p, m, di, s);
    return k8 ? launch<8, true>(p, m, di, s) : launch<8, false>(p, m, di, s);
}

}  // namespace hc
