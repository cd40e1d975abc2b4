"""64-bit forms of the norm and the embedding, and bounds on binary32's errors in them.

The bounds follow a value through the operations that make it: u = 2^-24 is half a step of
binary32, a sum of which no number passes through more than K additions is off by K u times the sum
of its terms' magnitudes, and the last step rounds to the rows' type.
"""
import torch

U32 = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half a step of the numbers below the type's normal ones
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def chain(d):
    """Additions that a term of a row's sum passes through: a row of d channels is shared by 32
    lanes at least, or by lanes with 32 channels each, whose sums meet in ten steps at most."""
    return d / 32 + 48


def norm(x, w, b, center, eps):
    """x [n, d], w, b [d] or None, all 64-bit -> y."""
    c = x - x.mean(1, keepdim=True) if center else x
    h = c / torch.sqrt(c.square().mean(1, keepdim=True) + eps)
    y = h if w is None else h * w
    return y if b is None else y + b


def _errors(x, center, eps):
    """h, r, and how far binary32's h and (relatively) r may be off."""
    k = chain(x.shape[1])
    mu = x.mean(1, keepdim=True) if center else torch.zeros_like(x[:, :1])
    dmu = (k + 2) * U32 * x.abs().mean(1, keepdim=True) if center else torch.zeros_like(mu)
    c = x - mu
    v = c.square().mean(1, keepdim=True)
    r = (v + eps) ** -0.5
    # the squares' sum, what the mean's error does to it, and their like; then 1 / sqrt to 2 steps
    off_v = (k + 6) * U32 * v + 2 * dmu * c.abs().mean(1, keepdim=True) + dmu.square()
    rel_r = 0.5 * off_v / (v + eps) + 6 * U32
    h = c * r
    off_h = h.abs() * (rel_r + 4 * U32) + dmu * r
    return h, r, off_h, rel_r


def norm_bound(x, w, b, center, eps, dtype):
    h, _, off_h, _ = _errors(x, center, eps)
    y = norm(x, w, b, center, eps)
    wa = 1.0 if w is None else w.abs()
    off = off_h * wa + 2 * U32 * (h.abs() * wa + y.abs())
    return off * 1.01 + (1 + 1e-3) * HALF[dtype] * y.abs() + TINY[dtype]


def norm_backward(dy, x, w, center, eps):
    """-> dx, dweight, dbias."""
    mu = x.mean(1, keepdim=True) if center else 0.0
    c = x - mu
    r = (c.square().mean(1, keepdim=True) + eps) ** -0.5
    h = c * r
    g = dy if w is None else dy * w
    dx = g - h * (g * h).mean(1, keepdim=True)
    if center:
        dx = dx - g.mean(1, keepdim=True)
    return r * dx, (dy * h).sum(0), dy.sum(0)


def norm_backward_bound(dy, x, w, center, eps, dtype):
    n, d = x.shape
    k = chain(d)
    h, r, off_h, rel_r = _errors(x, center, eps)
    g = dy if w is None else dy * w
    dx, dw, db = norm_backward(dy, x, w, center, eps)
    c1 = g.mean(1, keepdim=True) if center else torch.zeros_like(r)
    off1 = (k + 3) * U32 * g.abs().mean(1, keepdim=True) if center else torch.zeros_like(r)
    c2 = (g * h).mean(1, keepdim=True)
    off2 = (k + 5) * U32 * (g * h).abs().mean(1, keepdim=True) + \
        (g.abs() * off_h).mean(1, keepdim=True)
    off = r * (off1 + h.abs() * off2 + c2.abs() * off_h +
               4 * U32 * (g.abs() + c1.abs() + (h * c2).abs())) + dx.abs() * rel_r
    off = off * 1.01 + (1 + 1e-3) * HALF[dtype] * dx.abs() + TINY[dtype]
    # a block adds up its rows one by one, and up to 608 blocks' sums are added up by 32 threads
    kw = min(n, n / 64 + 400) + 16
    off_w = kw * U32 * (dy * h).abs().sum(0) + (dy.abs() * off_h).sum(0)
    return off, off_w * 1.01 + 1e-44, kw * U32 * dy.abs().sum(0) + 1e-44


def embed_backward(ids, dx, vocab, scale):
    """ids [n] int64, dx [n, hc, d] 64-bit -> the sums and the sums of their magnitudes."""
    ok = (ids >= 0) & (ids < vocab)
    out = torch.zeros(2, vocab, dx.shape[2], dtype=torch.float64)
    out[0].index_add_(0, ids[ok], dx[ok].sum(1))
    out[1].index_add_(0, ids[ok], dx[ok].abs().sum(1))
    return out[0] * scale, out[1] * abs(scale)


def embed_chain(n):
    """Additions a gradient passes through: 8 copies of 32 tokens, then an eighth of the pieces of
    its id, 8 partial sums, the scale.  n / 8 allows for pieces of single tokens; the library's have
    four or more (embed_backward_bound)."""
    return 8 * 32 + n / 8 + 16


def embed_backward_bound(n, want, mag, dtype, added=False):
    """How far a table's gradient, `want` in 64 bits, may be off where n tokens' gradients, of
    magnitudes that sum to `mag`, are added up: 8 copies of the 32 tokens of a piece, then of the
    n / 4 pieces that an id has at most (a piece has four tokens or more) an eighth, then 8 partial
    sums and the scale; added to what was there in one more step; rounded to the type once."""
    off = (8 * 32 + n / 32 + 16) * U32 * mag + (U32 * want.abs() if added else 0)
    return off * 1.01 + (1 + 1e-3) * HALF[dtype] * want.abs() + TINY[dtype]


def check_embed_backward(got, base, ids, dx, vocab, scale, dtype, seed=0):
    """A table's gradient `got` (with `base`, added to that) against the 64-bit sums, element by
    element, and against differences of the 64-bit lookup along directions in which the gradient's
    terms do not cancel: all of it, and one row.  What a difference may be off by follows from the
    bound of the elements alone, and not from `got`."""
    got, dx = got.detach().cpu().double(), dx.detach().cpu().double()
    ids = ids.cpu().long()
    want, mag = embed_backward(ids, dx, vocab, scale)
    total = want if base is None else want + base.cpu().double()
    bound = embed_backward_bound(ids.numel(), total, mag, dtype, base is not None)
    assert torch.all((got - total).abs() <= bound), float(((got - total).abs() - bound).max())
    if base is not None:
        got = got - base.cpu().double()
    ok = (ids >= 0) & (ids < vocab)
    g = torch.Generator().manual_seed(seed)
    table = torch.randn(want.shape, generator=g, dtype=torch.float64)

    def loss(t):
        return (scale * t[ids[ok]] * dx[ok].sum(1)).sum()

    along = want.sign() * (0.5 + torch.rand(want.shape, generator=g, dtype=torch.float64))
    one = torch.zeros_like(along)
    row = int(mag.sum(1).argmax())
    one[row] = along[row]
    for u in (along, one):
        diff = (loss(table + u) - loss(table - u)) / 2      # linear: any step will do
        slack = 1e-12 * ((table.abs() + u.abs()) * mag).sum()
        assert abs(float((got * u).sum() - diff)) <= float((bound * u.abs()).sum() + slack)
