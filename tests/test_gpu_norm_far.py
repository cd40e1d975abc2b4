"""Layer norm and its gradients of rows whose mean is thousands of deviations away, in fp32 (GPU).

The bounds hold no term of half a step of the mean times 1 / sqrt(variance): they follow the row's
numbers about a number p that is subtracted from them exactly (both lie within a factor of two of
one another), and what the mean differs from p by is taken off as a number of its own."""
import pytest
import torch

import rows_reference as ref

pytestmark = pytest.mark.gpu
EPS = 1e-5
# every way in which rows are shared out
WIDTHS = [64, 520, 1000, 5120, 8192, 8200, 12296, 20480, 20488, 32776, 65544]


@pytest.fixture(scope="module")
def hc():
    import sinkhorn_mixing_gb300 as lib
    lib.lib()
    yield lib
    assert lib.hc_device_error(clear=True) == 0


# few rows and more than there are SMs: wide rows go to blocks of another size
ROWS = [7, 160]


def case(rows, d):
    g = torch.Generator().manual_seed(d)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    mean = torch.tensor([1000.0, -1000.0, 3.0, 777.7, -0.01, 65.3, 1001.0])
    mean = mean.repeat(rows // 7 + 1)[:rows, None]
    return mean + 0.05 * r(rows, d), r(rows, d) * 2.0 ** -6, 1 + 0.5 * r(d), r(d)


def errors(x):
    """h, r, and how far binary32's h and (relatively) r may be off.  p is off the mean by a
    deviation at most, or by what a sum of the row is rounded by; a sum's terms pass through
    ref.chain(d) additions at most."""
    k, u = ref.chain(x.shape[1]), ref.U32
    c = x - x.mean(1, keepdim=True)
    v = c.square().mean(1, keepdim=True)
    r = (v + EPS) ** -0.5
    off_p = 1.01 * v.sqrt() + (k + 2) * u * x.abs().mean(1, keepdim=True)
    # the mean of x - p: its sum, and the rounding of a difference of numbers of unlike size
    dmu = (k + 4) * u * (c.abs().mean(1, keepdim=True) + off_p)
    off_v = (k + 6) * u * (v + off_p.square()) + 2 * off_p * dmu + dmu.square()
    rel_r = 0.5 * off_v / (v + EPS) + 6 * u
    h = c * r
    return h, r, h.abs() * rel_r + dmu * r + 4 * u * (c.abs() + 2 * off_p) * r, rel_r


def within(got, want, bound):
    worst = float(((got.cpu().double() - want).abs() / bound).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("d", WIDTHS)
def test_norm(hc, d, rows):
    x, _, w, b = case(rows, d)
    y = hc.hc_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS, center=True)
    x, w, b = x.double(), w.double(), b.double()
    h, _, off_h, _ = errors(x)
    want = ref.norm(x, w, b, True, EPS)
    within(y, want, 1.01 * (off_h * w.abs() + 3 * ref.U32 * ((h * w).abs() + want.abs())))


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("d", WIDTHS)
def test_norm_backward(hc, d, rows):
    x, dy, w, _ = case(rows, d)
    got = hc.hc_norm_backward(dy.cuda(), x.cuda(), w.cuda(), eps=EPS, center=True, want_dbias=True)
    x, dy, w = x.double(), dy.double(), w.double()
    h, r, off_h, rel_r = errors(x)
    g, k, u = dy * w, ref.chain(d), ref.U32
    dx, dw, db = ref.norm_backward(dy, x, w, True, EPS)
    c1, c2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    off1 = (k + 3) * u * g.abs().mean(1, keepdim=True)
    # mean(g h): the sum of g (x - p), whose terms are h's and the mean's distance from p
    off_p = 1.01 / r + (k + 2) * u * x.abs().mean(1, keepdim=True)
    off2 = (k + 5) * u * (g.abs() * (h.abs() + off_p * r)).mean(1, keepdim=True) + \
        (g.abs() * off_h).mean(1, keepdim=True) + off_p * r * off1
    off = r * (off1 + h.abs() * off2 + c2.abs() * off_h +
               5 * u * (g.abs() + c1.abs() + (h * c2).abs())) + dx.abs() * rel_r
    within(got[0], dx, 1.01 * off + 2 * u * dx.abs())
    adds = rows + 16
    within(got[1], dw, 1.01 * (adds * u * (dy * h).abs().sum(0) + (dy.abs() * off_h).sum(0)))
    within(got[2], db, adds * u * dy.abs().sum(0))
