"""The training operators in 64 bits, from their definitions (test infrastructure).

Gradients come from automatic differentiation of the forward definitions in
float64, apart from any formula the kernels use; kept tensors come from
integer arithmetic on bit patterns and a table of the e4m3 numbers.
"""
import numpy as np
import torch

U32 = 2.0 ** -24   # binary32's unit roundoff
UBF = 2.0 ** -8    # half a bf16 step, relative


# ------------------------------------------------------- rows kept in 8 bits

def e4m3_values():
    """The 256 codes' values: sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7F and 0xFF
    are NaN, and there is no infinity."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if c & 0x7F == 0x7F else (-a if c & 0x80 else a)
    return v


def checkpoint(bits):
    """codes, scales of rows of bf16 bit patterns (uint16 [rows, d])."""
    rows, d = bits.shape
    nblk = -(-d // 32)
    mag = np.zeros((rows, nblk * 32), np.int64)
    mag[:, :d] = bits & 0x7FFF
    bad = mag >= 0x7F80
    big = np.where(bad, 0, mag).reshape(rows, nblk, 32).max(2)
    scales = np.maximum(1, (big >> 7) - 8 + ((big & 0x7F) > 0x60))
    value = np.where(bad[:, :d], 0, np.uint32(0) + (bits & 0x7FFF)).astype(np.uint32) << 16
    value = value.view(np.float32).astype(np.float64)
    over = value / np.exp2(np.repeat(scales, 32, 1)[:, :d].astype(np.float64) - 127)
    grid = e4m3_values()[:127]                      # the magnitudes, ascending
    hi = np.clip(np.searchsorted(grid, over), 0, 126)
    lo = np.maximum(hi - 1, 0)
    below, above = over - grid[lo], grid[hi] - over
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    last = np.repeat(scales, 32, 1)[:, :d] == 247   # 256 * 2^120 is no bf16 number, 240 * 2^120 is
    code = np.where(last, np.minimum(code, 0x77), code)
    code = np.where(bits & 0x8000, code | 0x80, code)
    code = np.where(bad[:, :d], 0x7F, code)
    return code.astype(np.uint8), scales.astype(np.uint8)


def values(kept):
    """A kept tensor's numbers in float64 on the CPU."""
    if isinstance(kept, torch.Tensor):
        return kept.detach().cpu().double()
    codes, scales = kept
    c = codes.detach().cpu().view(torch.uint8).numpy()
    s = scales.detach().cpu().numpy().astype(np.float64)
    s = np.repeat(np.exp2(s - 127), 32, -1)[..., :c.shape[-1]]
    return torch.from_numpy(e4m3_values()[c] * s)


# ----------------------------------------------------------------- forward

def split(z, hc, iters, eps):
    pre = torch.sigmoid(z[:, :hc]) + eps
    post = 2 * torch.sigmoid(z[:, hc:2 * hc])
    c = torch.softmax(z[:, 2 * hc:].unflatten(1, (hc, hc)), 2) + eps
    c = c / (c.sum(1, keepdim=True) + eps)
    for _ in range(iters - 1):
        c = c / (c.sum(2, keepdim=True) + eps)
        c = c / (c.sum(1, keepdim=True) + eps)
    return pre, post, c


def mixes(x, w, norm_eps):
    v = x.flatten(1)
    return (v @ w.t()) * (v.square().mean(1, keepdim=True) + norm_eps) ** -0.5


def logits(m, scale, base, hc):
    return torch.cat([m[:, :hc] * scale[0], m[:, hc:2 * hc] * scale[1], m[:, 2 * hc:] * scale[2]],
                     1) + base


def mixes_pre(x, w, scale, base, iters, eps, norm_eps):
    hc = x.shape[1]
    m = mixes(x, w, norm_eps)
    pre, post, comb = split(logits(m, scale, base, hc), hc, iters, eps)
    return torch.einsum("nj,njc->nc", pre, x), pre, post, comb, m


def post(out, residual, post_, comb):
    return torch.einsum("nk,nc->nkc", post_, out) + torch.einsum("njk,njc->nkc", comb, residual)


# --------------------------------------------------------------- gradients

def post_backward(dy, out, residual, post_, comb):
    """dout, dpost, dcomb, dresidual, and each one's sum of magnitudes of its terms."""
    leaves = [t.clone().requires_grad_() for t in (out, post_, comb, residual)]
    grads = torch.autograd.grad(post(leaves[0], leaves[3], leaves[1], leaves[2]), leaves, dy)
    leaves = [t.abs().requires_grad_() for t in (out, post_, comb, residual)]
    mags = torch.autograd.grad(post(leaves[0], leaves[3], leaves[1], leaves[2]), leaves, dy.abs())
    return grads, mags


def mixes_pre_backward(dy, x, m, w, scale, base, dpost, dcomb, dstream, iters, eps, norm_eps):
    """dx, dw, dscale, dbase; then du and the magnitudes |terms| that make up dx and dw.
    m: the forward pass's mix numbers, whose values enter where the definition has them."""
    n, hc, d = x.shape
    x = x.clone().requires_grad_()
    scale, base = scale.clone().requires_grad_(), base.clone().requires_grad_()
    r = (x.flatten(1).square().mean(1, keepdim=True) + norm_eps) ** -0.5
    u = (m / r).detach().requires_grad_()
    pre, post_, comb = split(logits(r * u, scale, base, hc), hc, iters, eps)
    y = torch.einsum("nj,njc->nc", pre, x)
    past = torch.einsum("njk,njc->nkc", comb.detach(), x)
    ds = torch.zeros(n, hc, d, dtype=torch.float64) if dstream is None else dstream
    gx, du, gs, gb = torch.autograd.grad((y, past, post_, comb), (x, u, scale, base),
                                         (dy, ds, dpost, dcomb))
    xv = x.detach()
    dx = gx + (du @ w).view(n, hc, d)
    dw = du.t() @ xv.flatten(1)
    q = (du * u).sum(1).abs() * r.detach()[:, 0] ** 2 / (hc * d)
    proj = (du.abs() @ w.abs()).view(n, hc, d)
    rest = (pre[..., None] * dy[:, None].abs() + q[:, None, None] * xv.abs() +
            torch.einsum("njk,nkc->njc", comb, ds.abs())).detach()
    return (dx, dw, gs, gb), dict(du=du, proj=proj, rest=rest,
                                  dw=du.abs().t() @ xv.flatten(1).abs())


def split_tolerance(iters):
    """Relative error (2-norm) allowed to what passes backward through the split in binary32:
    2 iters - 1 steps forth, as many back, each with at most 16 roundings (sums of up to 8 terms,
    a reciprocal, products).  A step back is the divided projection (g - <g, c'> 1) / den with
    den near 1, of norm near 1, so the steps' errors add up and do not multiply."""
    return (4 * iters + 4) * 16 * U32
