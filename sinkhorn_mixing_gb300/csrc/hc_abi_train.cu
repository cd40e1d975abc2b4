// hc_abi_train.cu -- the C entry points of the training operators: rows kept in
// 8 bits, and gradients.  Host-side argument validation and launch; nothing
// here allocates memory.
#include "hc_check.h"
#include "hc_internal.h"
#include "hc_kept.cuh"
#include "hc_pre_bwd.h"

using namespace hc::check;

namespace {

// rows of d channels: the byte counts stay inside int64
hc_status check_rows(int64_t rows, int64_t d) {
    if (rows < 0 || d <= 0) return HC_ERR_INVALID_ARG;
    if (d % 8 != 0) return HC_ERR_MISALIGNED;
    if (d > (int64_t(1) << 24) || rows > (int64_t(1) << 58) / d) return HC_ERR_UNSUPPORTED;
    return HC_OK;
}

hc_status check_tokens(int64_t n, int hc, int64_t d) {
    const hc_status st = check_shape(n, hc, d);
    return st != HC_OK ? st : check_rows(n * hc, d);
}

// scale bytes are read and written one by one: any address will do
hc_status scales_ok(const uint8_t *p) { return p == nullptr ? HC_ERR_INVALID_ARG : HC_OK; }

uint64_t scale_bytes(uint64_t rows, int64_t d) { return rows * (uint64_t)hc::kept_blocks(d); }

// A kept tensor's two ranges: bf16 rows (no scales), or codes and scales.
Range kept_data(const void *p, const uint8_t *scales, uint64_t rows, int64_t d) {
    return rng(p, rows * (uint64_t)d * (scales ? 1 : 2));
}
Range kept_scales(const uint8_t *scales, uint64_t rows, int64_t d) {
    return scales ? rng(scales, scale_bytes(rows, d)) : Range{0, 0};
}

}  // namespace

extern "C" {

hc_status hc_checkpoint(int64_t rows, int64_t d, const uint16_t *x, uint8_t *codes,
                        uint8_t *scales, hc_stream_t stream) {
    hc_status st = check_rows(rows, d);
    if (st != HC_OK) return st;
    if (rows == 0) return HC_OK;
    if ((st = ptrs_ok({x, codes})) != HC_OK || (st = scales_ok(scales)) != HC_OK) return st;
    const uint64_t el = (uint64_t)rows * d;
    if (!disjoint({rng(codes, el), rng(scales, scale_bytes(rows, d))}, {rng(x, el * 2)}))
        return HC_ERR_INVALID_ARG;
    hc::DeviceInfo di;
    if (hc::device_info(&di) != cudaSuccess) return cuda_failed();
    return from_cuda(hc::launch_checkpoint(rows, d, x, codes, scales, di,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

hc_status hc_restore(int64_t rows, int64_t d, const uint8_t *codes, const uint8_t *scales,
                     uint16_t *x, hc_stream_t stream) {
    hc_status st = check_rows(rows, d);
    if (st != HC_OK) return st;
    if (rows == 0) return HC_OK;
    if ((st = ptrs_ok({codes, x})) != HC_OK || (st = scales_ok(scales)) != HC_OK) return st;
    const uint64_t el = (uint64_t)rows * d;
    if (!disjoint({rng(x, el * 2)}, {rng(codes, el), rng(scales, scale_bytes(rows, d))}))
        return HC_ERR_INVALID_ARG;
    hc::DeviceInfo di;
    if (hc::device_info(&di) != cudaSuccess) return cuda_failed();
    return from_cuda(hc::launch_restore(rows, d, hc::Kept{codes, scales}, x, di,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

hc_status hc_pre_restore(int64_t n, int hc, int64_t d, const uint8_t *codes,
                         const uint8_t *scales, const float *pre, uint16_t *y,
                         hc_stream_t stream) {
    hc_status st = check_tokens(n, hc, d);
    if (st != HC_OK) return st;
    if (n == 0) return HC_OK;
    if ((st = ptrs_ok({codes, pre, y})) != HC_OK || (st = scales_ok(scales)) != HC_OK) return st;
    const uint64_t rows = (uint64_t)n * hc;
    if (!disjoint({rng(y, (uint64_t)n * d * 2)},
                  {rng(codes, rows * d), rng(scales, scale_bytes(rows, d)), rng(pre, rows * 4)}))
        return HC_ERR_INVALID_ARG;
    hc::DeviceInfo di;
    if (hc::device_info(&di) != cudaSuccess) return cuda_failed();
    return from_cuda(hc::launch_pre_restore(n, hc, d, hc::Kept{codes, scales}, pre, y, di,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

hc_status hc_post_checkpoint(int64_t n, int hc, int64_t d, const uint16_t *out,
                             const uint16_t *residual, const float *post, const float *comb,
                             uint16_t *y, uint8_t *codes, uint8_t *scales, hc_stream_t stream) {
    hc_status st = check_tokens(n, hc, d);
    if (st != HC_OK) return st;
    if (n == 0) return HC_OK;
    if ((st = ptrs_ok({out, residual, post, comb, y, codes})) != HC_OK ||
        (st = scales_ok(scales)) != HC_OK)
        return st;
    const uint64_t rows = (uint64_t)n * hc, el = rows * d;
    const Range ry = rng(y, el * 2), rr = rng(residual, el * 2), rc = rng(codes, el),
                rs = rng(scales, scale_bytes(rows, d));
    const bool in_place = (const void *)y == (const void *)residual;
    if (!in_place && overlap(ry, rr)) return HC_ERR_INVALID_ARG;
    if (!disjoint({ry, rc, rs}, {rng(out, (uint64_t)n * d * 2), rng(post, rows * 4),
                                 rng(comb, rows * hc * 4)}) ||
        !disjoint({rc, rs}, {rr}))
        return HC_ERR_INVALID_ARG;
    hc::DeviceInfo di;
    if (hc::device_info(&di) != cudaSuccess) return cuda_failed();
    return from_cuda(hc::launch_post_checkpoint(n, hc, d, out, residual, post, comb, y, codes,
                                                scales, di,
                                                reinterpret_cast<cudaStream_t>(stream)));
}

hc_status hc_post_backward(int64_t n, int hc, int64_t d, const uint16_t *dy, const void *out,
                           const uint8_t *out_scales, const void *residual,
                           const uint8_t *residual_scales, const float *post, const float *comb,
                           uint16_t *dout, float *dpost, float *dcomb, uint16_t *dresidual,
                           hc_stream_t stream) {
    hc_status st = check_tokens(n, hc, d);
    if (st != HC_OK) return st;
    if (n == 0) return HC_OK;
    if ((st = ptrs_ok({dy, out, residual, post, comb, dout, dpost, dcomb})) != HC_OK) return st;
    if (!al16(dresidual)) return HC_ERR_MISALIGNED;
    const uint64_t rows = (uint64_t)n * hc;
    const Range rg = rng(dy, rows * d * 2);
    const Range rres = dresidual ? rng(dresidual, rows * d * 2) : Range{0, 0};
    const Range rdo = rng(dout, (uint64_t)n * d * 2), rdp = rng(dpost, rows * 4),
                rdc = rng(dcomb, rows * hc * 4);
    if ((const void *)dresidual != (const void *)dy && overlap(rres, rg)) return HC_ERR_INVALID_ARG;
    if (!disjoint({rdo, rdp, rdc, rres},
                  {kept_data(out, out_scales, n, d), kept_scales(out_scales, n, d),
                   kept_data(residual, residual_scales, rows, d),
                   kept_scales(residual_scales, rows, d), rng(post, rows * 4),
                   rng(comb, rows * hc * 4)}) ||
        !disjoint({rdo, rdp, rdc}, {rg}))
        return HC_ERR_INVALID_ARG;
    hc::DeviceInfo di;
    if (hc::device_info(&di) != cudaSuccess) return cuda_failed();
    return from_cuda(hc::launch_post_backward(
        n, hc, d, dy, hc::Kept{out, out_scales}, hc::Kept{residual, residual_scales}, post, comb,
        dout, dpost, dcomb, dresidual, di, reinterpret_cast<cudaStream_t>(stream)));
}

size_t hc_mixes_pre_backward_bytes(int64_t n, int hc, int64_t d) {
    if (check_tokens(n, hc, d) != HC_OK || n == 0) return 0;
    return hc::pre_backward_bytes(n, hc, d);
}

hc_status hc_mixes_pre_backward(int64_t n, int hc, int64_t d, int iters, float eps, float norm_eps,
                                const uint16_t *dy, const void *x, const uint8_t *x_scales,
                                const float *mixes, const float *w_mix, const float *hc_scale,
                                const float *hc_base, const float *dpost, const float *dcomb,
                                const uint16_t *dstream, uint16_t *dx, float *dw_mix,
                                float *dscale, float *dbase, void *workspace,
                                size_t workspace_bytes, hc_stream_t stream) {
    hc_status st = check_tokens(n, hc, d);
    if (st != HC_OK) return st;
    if (iters < 1 || !finite_nonneg(eps) || !finite_nonneg(norm_eps)) return HC_ERR_INVALID_ARG;
    if (iters > hc::kBackwardMaxIters) return HC_ERR_UNSUPPORTED;
    const uint64_t mix = (uint64_t)(2 + hc) * hc, F = (uint64_t)hc * d;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (n == 0) {
        // no tokens: the parameters' gradients are zero, not left as they were
        if ((st = ptrs_ok({dw_mix, dscale, dbase})) != HC_OK) return st;
        if (!disjoint({rng(dw_mix, mix * F * 4), rng(dscale, 12), rng(dbase, mix * 4)}, {}))
            return HC_ERR_INVALID_ARG;
        cudaError_t e = cudaMemsetAsync(dw_mix, 0, mix * F * 4, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(dscale, 0, 12, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(dbase, 0, mix * 4, s);
        return from_cuda(e);
    }
    if ((st = ptrs_ok({dy, x, mixes, w_mix, hc_scale, hc_base, dpost, dcomb, dx, dw_mix, dscale,
                       dbase})) != HC_OK)
        return st;
    if (!al16(dstream)) return HC_ERR_MISALIGNED;
    if (workspace == nullptr || workspace_bytes < hc::pre_backward_bytes(n, hc, d))
        return HC_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return HC_ERR_MISALIGNED;
    const uint64_t rows = (uint64_t)n * hc;
    const Range rg = dstream ? rng(dstream, rows * d * 2) : Range{0, 0};
    const Range rdx = rng(dx, rows * d * 2), rdw = rng(dw_mix, mix * F * 4), rds = rng(dscale, 12),
                rdb = rng(dbase, mix * 4), rws = rng(workspace, workspace_bytes);
    if ((const void *)dx != (const void *)dstream && overlap(rdx, rg)) return HC_ERR_INVALID_ARG;
    if (!disjoint({rdx, rdw, rds, rdb, rws},
                  {rng(dy, (uint64_t)n * d * 2), kept_data(x, x_scales, rows, d),
                   kept_scales(x_scales, rows, d), rng(mixes, (uint64_t)n * mix * 4),
                   rng(w_mix, mix * F * 4), rng(hc_scale, 12), rng(hc_base, mix * 4),
                   rng(dpost, rows * 4), rng(dcomb, rows * hc * 4)}) ||
        !disjoint({rdw, rds, rdb, rws}, {rg}))
        return HC_ERR_INVALID_ARG;
    hc::DeviceInfo di;
    if (hc::device_info(&di) != cudaSuccess) return cuda_failed();
    hc::PreBackward p;
    p.n = n, p.d = d, p.hc = hc, p.iters = iters, p.eps = eps, p.norm_eps = norm_eps;
    p.dy = dy, p.x = hc::Kept{x, x_scales}, p.mixes = mixes, p.w = w_mix, p.scale = hc_scale;
    p.base = hc_base, p.dpost = dpost, p.dcomb = dcomb, p.dstream = dstream, p.dx = dx;
    p.dw = dw_mix, p.dscale = dscale, p.dbase = dbase;
    p.ws = static_cast<uint8_t *>(workspace);
    return from_cuda(hc::launch_pre_backward(p, di, s));
}

}  // extern "C"
