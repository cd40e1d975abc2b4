// hc_rownorm_bwd.cu -- gradients of the norm y = h w + b, h = (x - mu) r.
//
// With g = dy w, per row:
//   dx = r (g - mean(g) [layer norm] - h mean(g h))
// and over the rows dw = sum dy h, db = sum dy.
//
// The sums over rows: every block adds up the rows it has, in registers, and
// leaves one row of partial sums; k_norm_sum adds those up in a fixed order.
#include <algorithm>

#include "hc_rows.cuh"

namespace hc {
namespace {

constexpr int kStages = 3;         // rows a group has under way
constexpr int kRingThreads = 512;  // of a block at most: 128 registers each
constexpr int kParts = 304;        // rows of partial sums: two for each of a GB300's 152 SMs
constexpr int kLongChannels = 40;  // a thread's, of a row that does not fit the ring
constexpr int kLongRow = kLongChannels * kRingThreads;

// Rows of partial sums at most, by the width: up to four blocks an SM where rows are narrow,
// one for each SM of a GB300 where they are long.  Up to 10 MB for dweight and as much for
// dbias (12.5 MB each at 20,480 channels), but never less than a row of d floats each.
int64_t max_parts(int64_t rows, int64_t d) {
    int64_t m = (int64_t)kParts * 8192 / d;
    m = m > 2 * kParts ? 2 * kParts : m < 1 ? 1 : m;
    if (d <= kLongRow && m < kParts / 2) m = kParts / 2;
    return rows < m ? rows : m;
}

// So few rows that one block has them all: it writes dweight and dbias itself, and the call
// needs neither partial sums nor a second launch (18 us of the host's time through Python
// become 14).  A block takes about 1.2 us for the rows it has at a time; many blocks and the
// second launch take 4 to 5 us in all.
constexpr int kAloneSteps = 3;

// Vectors of a row that a thread has.
int ring_vecs(int64_t nv) {
    // four vectors a thread, or five, where a warp has the row; three in blocks where they do
    return row_vecs(nv, kRingThreads, nv <= 160 ? 5 : nv <= 3 * kRingThreads ? 3 : 4);
}
bool one_block(int64_t rows, int64_t nv) {
    return nv <= 4 * kRingThreads &&
           rows <= (int64_t)kAloneSteps * row_plan(nv, ring_vecs(nv), 1, 1).groups;
}

// What k_norm_stats leaves of a row, a float4 and a float.
size_t stats_bytes(int64_t rows) { return ((size_t)rows * 20 + 255) & ~(size_t)255; }

template <int E>
__device__ __forceinline__ void put_sums(float *row, int64_t v, const float a[E]) {
#pragma unroll
    for (int q = 0; q < E / 4; ++q)
        reinterpret_cast<float4 *>(row)[v * (E / 4) + q] =
            make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
}

// Rows of up to 4 x kRingThreads vectors, shared out as in the forward kernel: a group
// of threads has a row, each thread V vecs of it, copied to shared memory kStages - 1
// rows ahead.  A thread's channels are the same in every row, so their weights and
// the sums over the block's rows stay in its registers.  DB: dbias as well.
//
// A row takes one round of sums: x^2 and g x or, for layer norm, x - p, (x - p)^2, g
// and g (x - p) (see row_guess).  Behind the sums x and dy are read from shared memory
// again, or held packed where registers are left: RMS 292 us held, 296 read again; 16,384
// x 16384, four vectors a thread, x held 233, both 263, none 272; layer norm's sums leave
// none (302 us there, 435 held).  Warps with rows of their own hold both.
//
// The mean is p + delta and is not rounded to one number: h = (x - p) r - delta r, whose x - p
// is exact where p is near x (fp32, mean 1000, deviation 0.05: dw off by 3e-8 of 0.2, with one
// number 5e-5).
//
// 65,536 x 5120 in bf16 (2.01 GB) 292 us, 6.9 TB/s: a copy's rate.  Layer norm with a bias 379 us:
// 14 warps an SM (128 registers) issue in 60% of the slots.  131,072 x 128 20 us (5.0
// TB/s), 50,000 x 2048 in fp32 187 us (6.6 TB/s), the launch of k_norm_sum within.
template <int DT, bool CENTER, bool DB, int V, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kRingThreads : 256,
                                  BLOCK ? 1 : V < 3 || (V == 3 && !DB) ? 2 : 1)
    k_norm_backward(int64_t rows, int nv, int lg, float eps, const uint4 *dy0,
                    const uint4 *__restrict__ x0, const float *__restrict__ w, uint4 *dx0,
                    float *__restrict__ part_w, float *__restrict__ part_b) {
    constexpr int E = RowVec<DT>::E, NS = CENTER ? 4 : 2, SLOTS = 2 * V + (CENTER ? 1 : 0);
    constexpr bool HOLD_X = !BLOCK || !CENTER, HOLD_DY = !BLOCK || (!CENTER && V < 4);
    extern __shared__ uint4 ring[];
    __shared__ __align__(16) float red[2][NS][32];
    if (BLOCK) clear_red(&red[0][0][0], 2 * NS * 32);
    griddep_wait_then_release();
    const int lanes = BLOCK ? blockDim.x : 1 << lg;
    const int l = BLOCK ? threadIdx.x : threadIdx.x & (lanes - 1);
    const int groups = BLOCK ? 1 : 256 >> lg;
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t t = (int64_t)blockIdx.x * groups + (BLOCK ? 0 : threadIdx.x >> lg);
    const float inv_d = 1.0f / (float)(nv * E);
    auto slot = [&](int stage, int array, int i) {
        return ring + (stage * SLOTS + array * V + i) * blockDim.x + threadIdx.x;
    };
    auto copy = [&](int64_t row, int stage) {
        if (row < rows) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (l + i * lanes < nv) {
                    copy16_async(slot(stage, 0, i), x0 + row * nv + l + i * lanes);
                    copy16_async(slot(stage, 1, i), dy0 + row * nv + l + i * lanes);
                }
            if (CENTER) copy16_async(slot(stage, 2, 0), x0 + row * nv);  // for row_guess
        }
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) copy(t + k * step, k);
    uint64_t wk[V][E / 2], aw[V][E / 2], ab[DB ? V : 1][E / 2];  // pairs of channels
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float f[E];
        if (l + i * lanes < nv) row_params<E>(w, l + i * lanes, 1.0f, f);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            wk[i][e] = pack2(f[2 * e], f[2 * e + 1]);
            aw[i][e] = ab[DB ? i : 0][e] = 0;
        }
    }
    int at = 0, odd = 0;
    // a warp stays together until the last of its rows
    for (int64_t first = t - (BLOCK ? 0 : (threadIdx.x & 31) >> lg); first < rows;
         first += step, t += step) {
        copies_wait<kStages - 2>();
        copy(t + (kStages - 1) * step, at == 0 ? kStages - 1 : at - 1);
        const bool in = t < rows;
        float s[NS], mu = 0.0f, delta = 0.0f, var;
        uint64_t f[E / 2], g[E / 2];
        if (CENTER && in) mu = row_guess<DT>(*slot(at, 2, 0));
        uint4 xr[HOLD_X ? V : 1], gr[HOLD_DY ? V : 1];
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (in && l + i * lanes < nv) {
                if (HOLD_X) xr[HOLD_X ? i : 0] = *slot(at, 0, i);
                if (HOLD_DY) gr[HOLD_DY ? i : 0] = *slot(at, 1, i);
            }
        auto read = [&](int i) {
            row_pairs<DT>(HOLD_X ? xr[HOLD_X ? i : 0] : *slot(at, 0, i), f);
            row_pairs<DT>(HOLD_DY ? gr[HOLD_DY ? i : 0] : *slot(at, 1, i), g);
        };
        auto sums = [&]() {
            uint64_t sq = 0, sgc = 0, sg = 0, sc = 0;
            const uint64_t minus_p = pack2(-mu, -mu);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (in && l + i * lanes < nv) {
                    read(i);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        const uint64_t c = CENTER ? fadd2(f[e], minus_p) : f[e];
                        const uint64_t gw = fmul2(g[e], wk[i][e]);
                        ffma2(sq, c, c);
                        ffma2(sgc, gw, c);
                        if (CENTER) sc = fadd2(sc, c), sg = fadd2(sg, gw);
                    }
                }
            s[0] = sum2(sq), s[1] = sum2(sgc);
            if (CENTER) s[NS - 2] = sum2(sc), s[NS - 1] = sum2(sg);
            group_sum<BLOCK, NS>(s, lg, red[odd]);
            odd ^= 1;
            var = s[0] * inv_d;
            if (CENTER) {
                delta = s[NS - 2] * inv_d;
                var = row_variance(var, delta);
            }
        };
        sums();
        if (CENTER) {
            // the same for all of a block; all of a warp go along, in vain but for those in need
            const bool again = row_again(var, delta);
            if (BLOCK ? again : __any_sync(0xFFFFFFFFu, again)) {
                if (again) mu += delta;
                sums();
            }
        }
        const float r = rsqrtf(var + eps);
        // mean(g h); 0 with r, whatever sum g x came to in a row too large for its squares
        const float c1 = CENTER ? s[NS - 1] * inv_d : 0.0f;
        const float gc = CENTER ? fmaf(-delta, c1, s[1] * inv_d) : s[1] * inv_d;
        const float c2 = r == 0.0f ? 0.0f : gc * r;
        const float rc1 = -c1 * r, rc2 = -c2 * r, dr = r == 0.0f ? 0.0f : -delta * r;
        const uint64_t rr = pack2(r, r), minus_mu = pack2(-mu, -mu), minus_dr = pack2(dr, dr),
                       minus_rc1 = pack2(rc1, rc1), minus_rc2 = pack2(rc2, rc2);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (in && l + i * lanes < nv) {
                read(i);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    const uint64_t h = CENTER ? ffma2_of(fadd2(f[e], minus_mu), rr, minus_dr)
                                              : fmul2(f[e], rr);
                    ffma2(aw[i][e], g[e], h);
                    if (DB) ab[DB ? i : 0][e] = fadd2(ab[DB ? i : 0][e], g[e]);
                    const uint64_t gw = fmul2(g[e], wk[i][e]);
                    f[e] = ffma2_of(h, minus_rc2,
                                    CENTER ? ffma2_of(gw, rr, minus_rc1) : fmul2(gw, rr));
                }
                st_stream(dx0 + t * nv + l + i * lanes, row_from_pairs<DT>(f));
            }
        at = at + 1 == kStages ? 0 : at + 1;
    }
    const int64_t d = (int64_t)nv * E;
    if (part_w != nullptr) part_w += blockIdx.x * d;
    if (DB && part_b != nullptr) part_b += blockIdx.x * d;
    float sw[E], sb[E];
    if (BLOCK) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (l + i * lanes < nv) {
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    unpack2(aw[i][e], sw[2 * e], sw[2 * e + 1]);
                    if (DB) unpack2(ab[DB ? i : 0][e], sb[2 * e], sb[2 * e + 1]);
                }
                if (part_w != nullptr) put_sums<E>(part_w, l + i * lanes, sw);
                if (DB && part_b != nullptr) put_sums<E>(part_b, l + i * lanes, sb);
            }
        return;
    }
    // the sums of a warp's groups, then of the block's warps, in the ring's memory
    copies_wait<0>();
    __syncthreads();
    float *buf = reinterpret_cast<float *>(ring);
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            unpack2(aw[i][e], sw[2 * e], sw[2 * e + 1]);
            if (DB) unpack2(ab[DB ? i : 0][e], sb[2 * e], sb[2 * e + 1]);
        }
#pragma unroll
        for (int k = 0; k < 5; ++k)
            if (k >= lg)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    sw[e] += __shfl_xor_sync(0xFFFFFFFFu, sw[e], 1 << k);
                    if (DB) sb[e] += __shfl_xor_sync(0xFFFFFFFFu, sb[e], 1 << k);
                }
        if ((int)(threadIdx.x & 31) < lanes && l + i * lanes < nv) {
            put_sums<E>(buf + warp * d, l + i * lanes, sw);
            if (DB) put_sums<E>(buf + (8 + warp) * d, l + i * lanes, sb);
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < (int)d; c += 256) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            a += buf[q * d + c];
            if (DB) b += buf[(8 + q) * d + c];
        }
        if (part_w != nullptr) part_w[c] = a;
        if (DB && part_b != nullptr) part_b[c] = b;
    }
}

// Rows of up to kLongRow channels that do not fit the ring: a block of kRingThreads has a row,
// reads it for the sums and, from L2, again for the outputs, while the next row is on
// its way from HBM to L2.  The sums over the block's rows stay in registers as above.
// 8,192 x 20480 in fp32 372 to 386 us (6.4 TB/s), in bf16 242 (4.2 TB/s; of RMS 88 bytes a thread
// do not fit its 128 registers), layer norm with a bias 250.
template <int DT, bool CENTER, bool DB>
__global__ void __launch_bounds__(kRingThreads)
    k_norm_backward_long(int64_t rows, int nv, float eps, const uint4 *dy0,
                         const uint4 *__restrict__ x0, const float *__restrict__ w, uint4 *dx0,
                         float *__restrict__ part_w, float *__restrict__ part_b) {
    constexpr int E = RowVec<DT>::E, V = kLongChannels / E, NS = CENTER ? 4 : 2;
    __shared__ __align__(16) float red[2][NS][32];
    clear_red(&red[0][0][0], 2 * NS * 32);
    griddep_wait_then_release();
    const int l = threadIdx.x;
    const float inv_d = 1.0f / (float)(nv * E);
    uint64_t aw[V][E / 2], ab[DB ? V : 1][E / 2];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < E / 2; ++e) aw[i][e] = ab[DB ? i : 0][e] = 0;
    auto weights = [&](int v, uint64_t k[E / 2]) {
        float f[E];
        row_params<E>(w, v, 1.0f, f);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) k[e] = pack2(f[2 * e], f[2 * e + 1]);
    };
    int odd = 0;
    for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
        const uint4 *x = x0 + t * nv, *dy = dy0 + t * nv;
        uint64_t f[E / 2], g[E / 2], wk[E / 2];
        // TOGETHER: the loads are behind no branch (past the row's end a thread reads its first
        // vector for nothing), so that as many go out together as registers allow.  8,192 x
        // 20480: RMS in bf16 234 us in place of 282, but fp32 483 in place of 372 and layer norm
        // in bf16 322 in place of 246, whose registers the loads take from the sums.
        constexpr bool TOGETHER = !DB && E == 8;
        auto read = [&](int i, uint64_t a[E / 2], uint64_t b[E / 2], uint64_t c[E / 2]) {
            const int at = l + i * kRingThreads, v = !TOGETHER || at < nv ? at : l;
            row_pairs<DT>(__ldg(x + v), a);
            row_pairs<DT>(dy[v], b);
            weights(v, c);
        };
        float s[NS], mu = CENTER ? row_guess<DT>(__ldg(x)) : 0.0f, delta = 0.0f, var;
        for (int round = 0;; ++round) {
            uint64_t sq = 0, sgc = 0, sg = 0, sc = 0;
            const uint64_t minus_p = pack2(-mu, -mu);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool in = l + i * kRingThreads < nv;
                if (!TOGETHER && !in) break;
                read(i, f, g, wk);
                if (in)
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        const uint64_t c = CENTER ? fadd2(f[e], minus_p) : f[e];
                        const uint64_t gw = fmul2(g[e], wk[e]);
                        ffma2(sq, c, c);
                        ffma2(sgc, gw, c);
                        if (CENTER) sc = fadd2(sc, c), sg = fadd2(sg, gw);
                    }
            }
            s[0] = sum2(sq), s[1] = sum2(sgc);
            if (CENTER) s[NS - 2] = sum2(sc), s[NS - 1] = sum2(sg);
            block_sum<NS>(s, red[odd]);
            odd ^= 1;
            var = s[0] * inv_d;
            if (!CENTER) break;
            delta = s[NS - 2] * inv_d;
            var = row_variance(var, delta);
            if (round != 0 || !row_again(var, delta)) break;  // the same for all of the block
            mu += delta;
        }
        if (t + gridDim.x < rows) {
            // a line of 128 bytes for each eighth thread's vector
            const int64_t ahead = (int64_t)gridDim.x * nv;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = l + i * kRingThreads;
                if (v < nv && (l & 7) == 0) {
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(x + ahead + v));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(dy + ahead + v));
                }
            }
        }
        const float r = rsqrtf(var + eps);
        const float c1 = CENTER ? s[NS - 1] * inv_d : 0.0f;
        const float gc = CENTER ? fmaf(-delta, c1, s[1] * inv_d) : s[1] * inv_d;
        const float c2 = r == 0.0f ? 0.0f : gc * r;
        const float rc1 = -c1 * r, rc2 = -c2 * r, dr = r == 0.0f ? 0.0f : -delta * r;
        const uint64_t rr = pack2(r, r), minus_mu = pack2(-mu, -mu), minus_dr = pack2(dr, dr),
                       minus_rc1 = pack2(rc1, rc1), minus_rc2 = pack2(rc2, rc2);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = l + i * kRingThreads;
            if (!TOGETHER && v >= nv) break;
            read(i, f, g, wk);
            if (v < nv) {
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    const uint64_t h = CENTER ? ffma2_of(fadd2(f[e], minus_mu), rr, minus_dr)
                                              : fmul2(f[e], rr);
                    ffma2(aw[i][e], g[e], h);
                    if (DB) ab[DB ? i : 0][e] = fadd2(ab[DB ? i : 0][e], g[e]);
                    const uint64_t gw = fmul2(g[e], wk[e]);
                    f[e] = ffma2_of(h, minus_rc2,
                                    CENTER ? ffma2_of(gw, rr, minus_rc1) : fmul2(gw, rr));
                }
                st_stream(dx0 + t * nv + v, row_from_pairs<DT>(f));
            }
        }
    }
    const int64_t d = (int64_t)nv * E;
    part_w += blockIdx.x * d, part_b += blockIdx.x * d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = l + i * kRingThreads;
        if (v >= nv) break;
        float sw[E], sb[E];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            unpack2(aw[i][e], sw[2 * e], sw[2 * e + 1]);
            if (DB) unpack2(ab[DB ? i : 0][e], sb[2 * e], sb[2 * e + 1]);
        }
        put_sums<E>(part_w, v, sw);
        if (DB) put_sums<E>(part_b, v, sb);
    }
}

// Any width, first part: a row's mean as its sum gives it, r, mean(g) and mean(g h), and, of layer
// norm, the number that makes (x - mean) r h (see k_norm_wide).  Six blocks an SM: layer norm's
// sums in 16 bits took 44 registers, 4,096 x 20488 in bf16 175 us in place of 170.
template <int DT, bool CENTER>
__global__ void __launch_bounds__(256, CENTER && DT != HC_F32 ? 6 : 0)
    k_norm_stats(int64_t rows, int64_t nv, float eps, const uint4 *__restrict__ dy0,
                 const uint4 *__restrict__ x0, const float *__restrict__ w,
                 float4 *__restrict__ stats, float *__restrict__ rest) {
    constexpr int E = RowVec<DT>::E, NS = CENTER ? 2 : 1;
    __shared__ __align__(16) float red[3][2][32];
    clear_red(&red[0][0][0], 192);
    griddep_wait_then_release();
    const float inv_d = 1.0f / (float)(nv * E);
    for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
        const uint4 *x = x0 + t * nv, *dy = dy0 + t * nv;
        float mu = 0.0f, delta = 0.0f, var, f[E], g[E], wv[E];
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
        float q[NS];
        q[0] = q[NS - 1] = 0.0f;
        for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
            RowVec<DT>::get(x[v], f);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float a = f[e] - mu;
                q[0] = fmaf(a, a, q[0]);
                if (CENTER) q[NS - 1] += a;
            }
        }
        block_sum<NS>(q, red[1]);
        var = q[0] * inv_d;
        if (CENTER) {
            delta = q[NS - 1] * inv_d;
            var = row_variance(var, delta);
        }
        const float r = rsqrtf(var + eps), minus_dr = r == 0.0f ? 0.0f : -delta * r;
        float c[2] = {0.0f, 0.0f};
        for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
            RowVec<DT>::get(x[v], f);
            RowVec<DT>::get(dy[v], g);
            row_params<E>(w, v, 1.0f, wv);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float ge = g[e] * wv[e];
                c[0] += ge;
                c[1] = fmaf(ge, CENTER ? fmaf(f[e] - mu, r, minus_dr) : f[e] * r, c[1]);
            }
        }
        block_sum<2>(c, red[2]);
        if (threadIdx.x == 0) {
            stats[t] = make_float4(mu, r, CENTER ? c[0] * inv_d : 0.0f, c[1] * inv_d);
            if (CENTER) rest[t] = minus_dr;
        }
        __syncthreads();  // red is used again by the next row
    }
}

// Second part: a block has 128 vectors of a run of rows.
template <int DT, bool CENTER>
__global__ void __launch_bounds__(128)
    k_norm_grad(int64_t rows, int64_t nv, int64_t run, const uint4 *dy,
                const uint4 *__restrict__ x, const float *__restrict__ w,
                const float4 *__restrict__ stats, const float *__restrict__ rest, uint4 *dx,
                float *__restrict__ dw, float *__restrict__ db) {
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
        const float minus_dr = CENTER ? __ldg(rest + t) : 0.0f;
        float f[E], g[E];
        RowVec<DT>::get(x[t * nv + v], f);
        RowVec<DT>::get(dy[t * nv + v], g);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float h = CENTER ? fmaf(f[e] - st.x, st.y, minus_dr) : f[e] * st.y;
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

// out[c] = sum over the partial rows of part[p][c]: a block has 32 channels, and each
// of its 32 groups of 8 lanes every 32nd row.
__global__ void __launch_bounds__(256)
    k_norm_sum(int parts, int64_t d4, const float4 *__restrict__ part_w, float4 *__restrict__ dw,
               const float4 *__restrict__ part_b, float4 *__restrict__ db) {
    __shared__ float4 red[8][8];
    griddep_wait_then_release();
    const float4 *part = blockIdx.y == 0 ? part_w : part_b;
    float4 *out = blockIdx.y == 0 ? dw : db;
    if (out == nullptr) return;
    const int l = threadIdx.x & 7, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 8 + l;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < d4) {
#pragma unroll 8
        for (int p = threadIdx.x >> 3; p < parts; p += 32) {
            const float4 v = part[(int64_t)p * d4 + c];
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
    }
#pragma unroll
    for (int off = 8; off < 32; off <<= 1) {
        a.x += __shfl_xor_sync(0xFFFFFFFFu, a.x, off);
        a.y += __shfl_xor_sync(0xFFFFFFFFu, a.y, off);
        a.z += __shfl_xor_sync(0xFFFFFFFFu, a.z, off);
        a.w += __shfl_xor_sync(0xFFFFFFFFu, a.w, off);
    }
    if (lane < 8) red[warp][l] = a;
    __syncthreads();
    if (threadIdx.x < 8 && c < d4) {
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            const float4 v = red[i][l];
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
        out[c] = a;
    }
}

cudaError_t launch_sums(const RowNormBackward &p, int parts, const float *part_w,
                        const float *part_b, cudaStream_t s) {
    if (p.dweight == nullptr && p.dbias == nullptr) return cudaSuccess;
    const int64_t d4 = p.d / 4;
    return launch_overlapped(&k_norm_sum, dim3((unsigned)((d4 + 7) / 8), p.dbias ? 2u : 1u),
                             dim3(256), 0, s, parts, d4, reinterpret_cast<const float4 *>(part_w),
                             reinterpret_cast<float4 *>(p.dweight),
                             reinterpret_cast<const float4 *>(part_b),
                             reinterpret_cast<float4 *>(p.dbias));
}

template <int DT, bool CENTER, bool DB, int V, bool BLOCK>
cudaError_t launch_ring(const RowNormBackward &p, const RowPlan &plan, int64_t nv,
                        const DeviceInfo &di, cudaStream_t s) {
    static SmemState smem;
    static std::atomic<int> regs;
    auto *kernel = &k_norm_backward<DT, CENTER, DB, V, BLOCK>;
    constexpr int most = kStages * (2 * V + (CENTER ? 1 : 0)) * (BLOCK ? kRingThreads : 256) * 16;
    cudaError_t e = allow_smem(smem, reinterpret_cast<const void *>(kernel), most, di);
    if (e != cudaSuccess) return e;
    const bool alone = one_block(p.rows, nv);
    const int64_t want = (p.rows + plan.groups - 1) / plan.groups,
                  cap = (int64_t)di.sms * blocks_per_sm(kernel, regs, plan),
                  most_parts = max_parts(p.rows, p.d);
    const int parts = alone ? 1 : (int)std::min(want, std::min(cap, most_parts));
    float *part_w = alone ? p.dweight : reinterpret_cast<float *>(p.ws);
    float *part_b = alone ? p.dbias : part_w + (size_t)parts * p.d;
    e = launch_overlapped(kernel, dim3((unsigned)parts), dim3(plan.threads), plan.ring, s, p.rows,
                          (int)nv, plan.lg, p.eps, static_cast<const uint4 *>(p.dy),
                          static_cast<const uint4 *>(p.x), p.weight, static_cast<uint4 *>(p.dx),
                          part_w, part_b);
    return alone || e != cudaSuccess ? e : launch_sums(p, parts, part_w, part_b, s);
}

template <int DT, bool CENTER, bool DB, int V>
cudaError_t launch_ring(const RowNormBackward &p, int64_t nv, const DeviceInfo &di,
                        cudaStream_t s) {
    const RowPlan plan = row_plan(nv, V, 2 * V + (CENTER ? 1 : 0), kStages);
    return plan.lg == kBlockRow ? launch_ring<DT, CENTER, DB, V, true>(p, plan, nv, di, s)
                                : launch_ring<DT, CENTER, DB, V, false>(p, plan, nv, di, s);
}

template <int DT, bool CENTER, bool DB>
cudaError_t launch_ring(const RowNormBackward &p, int64_t nv, const DeviceInfo &di,
                        cudaStream_t s) {
    switch (ring_vecs(nv)) {
        case 1: return launch_ring<DT, CENTER, DB, 1>(p, nv, di, s);
        case 2: return launch_ring<DT, CENTER, DB, 2>(p, nv, di, s);
        case 3: return launch_ring<DT, CENTER, DB, 3>(p, nv, di, s);
        case 5:
            return launch_ring<DT, CENTER, DB, 5, false>(
                p, row_plan(nv, 5, 10 + (CENTER ? 1 : 0), kStages), nv, di, s);
        default: return launch_ring<DT, CENTER, DB, 4>(p, nv, di, s);
    }
}

template <int DT, bool CENTER, bool DB>
cudaError_t launch_long(const RowNormBackward &p, int64_t nv, const DeviceInfo &di,
                        cudaStream_t s) {
    const int parts = (int)std::min((int64_t)di.sms, max_parts(p.rows, p.d));
    float *part_w = reinterpret_cast<float *>(p.ws), *part_b = part_w + (size_t)parts * p.d;
    const cudaError_t e = launch_overlapped(
        &k_norm_backward_long<DT, CENTER, DB>, dim3((unsigned)parts), dim3(kRingThreads), 0, s,
        p.rows, (int)nv, p.eps, static_cast<const uint4 *>(p.dy), static_cast<const uint4 *>(p.x),
        p.weight, static_cast<uint4 *>(p.dx), part_w, part_b);
    return e != cudaSuccess ? e : launch_sums(p, parts, part_w, part_b, s);
}

template <int DT, bool CENTER>
cudaError_t launch(const RowNormBackward &p, const DeviceInfo &di, cudaStream_t s) {
    const int64_t nv = p.d / RowVec<DT>::E, cap = (int64_t)di.sms * 64;
    if (nv <= 4 * kRingThreads)
        return CENTER || p.dbias ? launch_ring<DT, CENTER, true>(p, nv, di, s)
                                 : launch_ring<DT, CENTER, CENTER>(p, nv, di, s);
    if (p.d <= kLongRow)
        return CENTER || p.dbias ? launch_long<DT, CENTER, true>(p, nv, di, s)
                                 : launch_long<DT, CENTER, CENTER>(p, nv, di, s);
    const uint4 *dy = static_cast<const uint4 *>(p.dy), *x = static_cast<const uint4 *>(p.x);
    float4 *stats = reinterpret_cast<float4 *>(p.ws);
    const int64_t most = max_parts(p.rows, p.d), run = (p.rows + most - 1) / most;
    const int parts = (int)((p.rows + run - 1) / run);
    float *rest = reinterpret_cast<float *>(stats + p.rows);
    float *part_w = reinterpret_cast<float *>(p.ws + stats_bytes(p.rows));
    float *part_b = part_w + (size_t)parts * p.d;
    cudaError_t e = launch_overlapped(&k_norm_stats<DT, CENTER>,
                                      dim3((unsigned)(p.rows < cap ? p.rows : cap)), dim3(256), 0,
                                      s, p.rows, nv, p.eps, dy, x, p.weight, stats, rest);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(&k_norm_grad<DT, CENTER>,
                          dim3((unsigned)((nv + 127) / 128), (unsigned)parts), dim3(128), 0, s,
                          p.rows, nv, run, dy, x, p.weight, (const float4 *)stats,
                          (const float *)rest, static_cast<uint4 *>(p.dx),
                          p.dweight ? part_w : nullptr, p.dbias ? part_b : nullptr);
    if (e != cudaSuccess) return e;
    return launch_sums(p, parts, part_w, part_b, s);
}

template <int DT>
cudaError_t launch(const RowNormBackward &p, const DeviceInfo &di, cudaStream_t s) {
    return p.center ? launch<DT, true>(p, di, s) : launch<DT, false>(p, di, s);
}

}  // namespace

size_t norm_backward_bytes(int64_t rows, int64_t d, int dtype) {
    if (one_block(rows, d * row_type_bytes(dtype) / 16)) return 0;
    return stats_bytes(rows) + (size_t)max_parts(rows, d) * (size_t)d * 8;
}

cudaError_t launch_norm_backward(const RowNormBackward &p, const DeviceInfo &di, cudaStream_t s) {
    return p.dtype == HC_BF16  ? launch<HC_BF16>(p, di, s)
           : p.dtype == HC_F16 ? launch<HC_F16>(p, di, s)
                               : launch<HC_F32>(p, di, s);
}

}  // namespace hc
