// hc_rownorm.cu -- the norm of rows: y = (x - mu) r * w + b, r = 1 / sqrt(v + eps),
// v the mean of (x - mu)^2, mu the row's mean (layer norm) or 0 (RMS norm).
//
// An HBM stream: each row is read once and written once.  65,536 x 5120 in bf16
// (1.34 GB) 216 us, 6.2 TB/s, 92% of a copy's rate, RMS and layer norm alike;
// 131,072 x 128 11.6 us, 5.8 TB/s; 32,768 x 1032 22.6 us, 6.0 TB/s; 64 x 5120 1.8 us.
#include "hc_rows.cuh"

namespace hc {
namespace {

constexpr int kStages = 3;         // rows a group has under way; 4: 226 us in place of 216
constexpr int kRingThreads = 512;  // of a block at most: 128 registers each
constexpr int kRingVecs = 4 * kRingThreads;

// Rows of up to kRingVecs vectors: a group of threads has a row, and each thread V vecs
// of it at most, which it copies to shared memory kStages - 1 rows ahead and reads
// once: the copies under way need no registers and no barrier.  A thread's channels
// are the same in every row, so it keeps their weights (and layer norm's biases) in
// registers: read again for each row they took twice the L1 traffic of the row
// itself (layer norm 278 us in place of 216).
template <int DT, bool CENTER, int V, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kRingThreads : 256, BLOCK ? 1 : V < 3 ? 3 : 2)
    k_norm(int64_t rows, int nv, int lg, float eps, const uint4 *x0, const float *__restrict__ w,
           const float *__restrict__ b, uint4 *y0) {
    constexpr int E = RowVec<DT>::E, NS = CENTER ? 2 : 1, SLOTS = V + (CENTER ? 1 : 0);
    constexpr bool KEEP_B = CENTER && V * E <= 32;
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
    auto slot = [&](int stage, int i) {
        return ring + (stage * SLOTS + i) * blockDim.x + threadIdx.x;
    };
    auto copy = [&](int64_t row, int stage) {
        if (row < rows) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (l + i * lanes < nv) copy16_async(slot(stage, i), x0 + row * nv + l + i * lanes);
            if (CENTER) copy16_async(slot(stage, V), x0 + row * nv);  // for row_guess
        }
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) copy(t + k * step, k);
    float wk[V][E], bk[KEEP_B ? V : 1][E];
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (l + i * lanes < nv) {
            row_params<E>(w, l + i * lanes, 1.0f, wk[i]);
            if (KEEP_B) row_params<E>(b, l + i * lanes, 0.0f, bk[i]);
        }
    int at = 0, odd = 0;
    // a warp stays together until the last of its rows
    for (int64_t first = t - (BLOCK ? 0 : (threadIdx.x & 31) >> lg); first < rows;
         first += step, t += step) {
        copies_wait<kStages - 2>();
        float mu = 0.0f, delta = 0.0f, var, f[V][E], s[NS];
        auto read = [&]() {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                const bool have = t < rows && l + i * lanes < nv;
                if (have) v = *slot(at, i);
                RowVec<DT>::get(v, f[i]);
                if (CENTER)
#pragma unroll
                    for (int e = 0; e < E; ++e) f[i][e] = have ? f[i][e] - mu : 0.0f;
            }
        };
        if (CENTER && t < rows) mu = row_guess<DT>(*slot(at, V));
        read();
        copy(t + (kStages - 1) * step, at == 0 ? kStages - 1 : at - 1);
        for (int round = 0;; ++round) {
            s[0] = s[NS - 1] = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    s[0] = fmaf(f[i][e], f[i][e], s[0]);
                    if (CENTER) s[NS - 1] += f[i][e];
                }
            group_sum<BLOCK, NS>(s, lg, red[odd]);
            odd ^= 1;
            var = s[0] * inv_d;
            if (!CENTER) break;
            delta = s[NS - 1] * inv_d;
            var = row_variance(var, delta);
            // the same for all of a block; all of a warp go along, in vain but for those in need
            const bool again = round == 0 && row_again(var, delta);
            if (BLOCK ? !again : !__any_sync(0xFFFFFFFFu, again)) break;
            if (again) mu += delta;
            read();
        }
        const float r = rsqrtf(var + eps), minus_dr = r == 0.0f ? 0.0f : -delta * r;
        if (t < rows) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (l + i * lanes < nv) {
                    float bv[E];
                    if (!KEEP_B) row_params<E>(b, l + i * lanes, 0.0f, bv);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        f[i][e] = fmaf(CENTER ? fmaf(f[i][e], r, minus_dr) : f[i][e] * r, wk[i][e],
                                       KEEP_B ? bk[i][e] : bv[e]);
                    st_stream(y0 + t * nv + l + i * lanes, RowVec<DT>::set(f[i]));
                }
            }
        }
        at = at + 1 == kStages ? 0 : at + 1;
    }
}

// Any width: a block a row, the row read once for each sum and once more for the
// output (from L1 or L2 after the first time).  8,192 x 20480 in bf16 114 us (5.9
// TB/s), layer norm with a bias 143 us; in one block's shared memory such a row left
// room for no other block, 117 and 183 us.
//
// A sum of numbers around a far mean is rounded to K u |mean|, which may be worth more
// than the row's deviation, and so is the mean that comes of it: with the squares about it
// goes a second sum, of what its numbers differ from it by (exact differences, as both are
// of one size), and takes the rest off (fp32, mean 1000, deviation 0.05: y is off by 2e-6 at
// most in place of 2e-3).  With that sum five blocks fit an SM, 157 us, six as it is bounded.  One
// round of sums about a guess, as k_norm has them, lost in spite of one reading less (160
// us): no row is copied ahead here, and all of its loads wait for the guess.
template <int DT, bool CENTER, int THREADS>
__global__ void __launch_bounds__(THREADS, CENTER && THREADS == 256 ? 6 : 0)
    k_norm_wide(int64_t rows, int64_t nv, float eps, const uint4 *x0, const float *__restrict__ w,
                const float *__restrict__ b, uint4 *y0) {
    constexpr int E = RowVec<DT>::E, NS = CENTER ? 2 : 1;
    __shared__ __align__(16) float red[3][32];
    clear_red(&red[0][0], 96);
    griddep_wait_then_release();
    const float inv_d = 1.0f / (float)(nv * E);
    for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
        const uint4 *x = x0 + t * nv;
        float mu = 0.0f, delta = 0.0f, var, f[E];
        if (CENTER) {
            float s[1] = {0.0f};
            for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
                RowVec<DT>::get(x[v], f);
#pragma unroll
                for (int e = 0; e < E; ++e) s[0] += f[e];
            }
            block_sum<1>(s, red);
            mu = s[0] * inv_d;
        }
        float q[NS];  // squares about mu and, in layer norm, what the mean differs from mu by
        q[0] = q[NS - 1] = 0.0f;
        for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
            RowVec<DT>::get(x[v], f);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float c = f[e] - mu;
                q[0] = fmaf(c, c, q[0]);
                if (CENTER) q[NS - 1] += c;
            }
        }
        block_sum<NS>(q, red + 1);
        var = q[0] * inv_d;
        if (CENTER) {
            delta = q[NS - 1] * inv_d;
            var = row_variance(var, delta);
        }
        const float r = rsqrtf(var + eps), minus_dr = r == 0.0f ? 0.0f : -delta * r;
        for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
            float wv[E], bv[E];
            RowVec<DT>::get(x[v], f);
            row_params<E>(w, v, 1.0f, wv);
            row_params<E>(b, v, 0.0f, bv);
#pragma unroll
            for (int e = 0; e < E; ++e)
                f[e] = fmaf(CENTER ? fmaf(f[e] - mu, r, minus_dr) : f[e] * r, wv[e], bv[e]);
            y0[t * nv + v] = RowVec<DT>::set(f);
        }
        __syncthreads();  // red is used again by the next row
    }
}

template <int DT, bool CENTER, int V, bool BLOCK>
cudaError_t launch_ring(const RowNorm &p, const RowPlan &plan, int64_t nv, const DeviceInfo &di,
                        cudaStream_t s) {
    static SmemState smem;
    static std::atomic<int> regs;
    auto *kernel = &k_norm<DT, CENTER, V, BLOCK>;
    constexpr int most = kStages * (V + (CENTER ? 1 : 0)) * (BLOCK ? kRingThreads : 256) * 16;
    const cudaError_t e = allow_smem(smem, reinterpret_cast<const void *>(kernel), most, di);
    if (e != cudaSuccess) return e;
    const int64_t want = (p.rows + plan.groups - 1) / plan.groups,
                  cap = (int64_t)di.sms * blocks_per_sm(kernel, regs, plan);
    return launch_overlapped(kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(plan.threads),
                             plan.ring, s, p.rows, (int)nv, plan.lg, p.eps,
                             static_cast<const uint4 *>(p.x), p.weight, p.bias,
                             static_cast<uint4 *>(p.y));
}

template <int DT, bool CENTER, int V>
cudaError_t launch_ring(const RowNorm &p, int64_t nv, const DeviceInfo &di, cudaStream_t s) {
    const RowPlan plan = row_plan(nv, V, V + (CENTER ? 1 : 0), kStages);
    return plan.lg == kBlockRow ? launch_ring<DT, CENTER, V, true>(p, plan, nv, di, s)
                                : launch_ring<DT, CENTER, V, false>(p, plan, nv, di, s);
}

template <int DT, bool CENTER, int THREADS>
cudaError_t launch_wide(const RowNorm &p, int64_t nv, const DeviceInfo &di, cudaStream_t s) {
    const int64_t cap = (int64_t)di.sms * 64;
    return launch_overlapped(&k_norm_wide<DT, CENTER, THREADS>,
                             dim3((unsigned)(p.rows < cap ? p.rows : cap)), dim3(THREADS), 0, s,
                             p.rows, nv, p.eps, static_cast<const uint4 *>(p.x), p.weight, p.bias,
                             static_cast<uint4 *>(p.y));
}

template <int DT, bool CENTER>
cudaError_t launch(const RowNorm &p, const DeviceInfo &di, cudaStream_t s) {
    const int64_t nv = p.d / RowVec<DT>::E;
    if (nv <= kRingVecs) {
        switch (row_vecs(nv, kRingThreads, 5)) {
            case 1: return launch_ring<DT, CENTER, 1>(p, nv, di, s);
            case 2: return launch_ring<DT, CENTER, 2>(p, nv, di, s);
            case 3: return launch_ring<DT, CENTER, 3>(p, nv, di, s);
            case 4: return launch_ring<DT, CENTER, 4>(p, nv, di, s);
            default: return launch_ring<DT, CENTER, 5>(p, nv, di, s);
        }
    }
    // No more rows than SMs: many threads for each.  100 x 20480 5.8 us in place of 7.1, layer norm
    // 7.5 and 8.5, 152 6.1 and 7.4; 153 rows, of which an SM has two in turn, 9.8 and 7.5, layer
    // norm 13.0 and 9.5, 304 11.2 and 8.6
    return p.rows <= di.sms ? launch_wide<DT, CENTER, 1024>(p, nv, di, s)
                            : launch_wide<DT, CENTER, 256>(p, nv, di, s);
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
