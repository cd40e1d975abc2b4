"""hc_norm and hc_norm_backward against their 64-bit forms (GPU)."""
import pytest
import torch

import rows_reference as ref

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [BF16, F16, F32]


@pytest.fixture(scope="module")
def hc():
    import sinkhorn_mixing_gb300 as lib
    lib.lib()
    yield lib
    assert lib.hc_device_error(clear=True) == 0


def case(rows, d, dtype, seed=0, weighted=True, biased=True):
    g = torch.Generator().manual_seed(rows * 31 + d + seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = (r(rows, d) * torch.exp(r(rows, 1)) + r(rows, 1)).to(dtype)
    dy = (r(rows, d) * 2.0 ** -6).to(dtype)
    return x, dy, 1 + 0.5 * r(d) if weighted else None, r(d) if biased else None


def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def f64(*ts):
    return [None if t is None else t.detach().cpu().double() for t in ts]


def within(got, want, bound, what):
    bad = ~((got.detach().cpu().double() - want).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((got.cpu().double() - want).abs().max()))


def check_norm(hc, x, w, b, center, eps, **kw):
    y = hc.hc_norm(*dev(x, w, b), eps=eps, center=center, **kw)
    assert y.dtype == x.dtype and y.shape == x.shape
    a = f64(x, w, b)
    within(y, ref.norm(*a, center, eps), ref.norm_bound(*a, center, eps, x.dtype), "y")


def check_backward(hc, dy, x, w, center, eps):
    got = hc.hc_norm_backward(*dev(dy, x, w), eps=eps, center=center, want_dbias=True)
    a = f64(dy, x, w)
    want = ref.norm_backward(*a, center, eps)
    bounds = ref.norm_backward_bound(*a, center, eps, x.dtype)
    for name, g, v, t in zip(("dx", "dweight", "dbias"), got, want, bounds):
        within(g, v, t, name)
    return got


# every way in which rows are shared out: rows narrower than a warp's vectors, rows of whole and of
# broken numbers of warps, rows that fill a block's registers and rows that do not fit them
WIDTHS = [8, 16, 24, 40, 64, 120, 128, 136, 256, 264, 512, 520, 1000, 1024, 1032, 1536, 2048, 2056,
          4096, 4104, 5120, 5128, 8192, 8200, 12288, 12296, 16384, 16392, 20480, 20488, 32768, 32776,
          65544]


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(hc, d, dtype, center):
    rows = 37 if d <= 2048 else 5
    x, dy, w, b = case(rows, d, dtype)
    check_norm(hc, x, w, b, center, 1e-5)
    check_backward(hc, dy, x, w, center, 1e-5)


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("rows,d", [(1, 8), (1, 5120), (2, 1000), (63, 5120), (151, 2048),
                                    (305, 1032), (613, 5120), (1001, 128), (2500, 1000),
                                    (70001, 16), (9999, 40), (1217, 8192), (700, 20480), (153, 16392),
                                    (400, 20488)])
def test_rows(hc, rows, d, center):
    for dtype in (BF16, F32):
        x, dy, w, b = case(rows, d, dtype, 1)
        check_norm(hc, x, w, b, center, 1e-20)
        check_backward(hc, dy, x, w, center, 1e-20)


@pytest.mark.parametrize("d", [40, 1000, 5120, 18440, 32776])
@pytest.mark.parametrize("center", [False, True])
def test_optional_parameters(hc, d, center):
    x, dy, w, b = case(33, d, BF16, 2)
    for ww, bb in ((None, None), (w, None), (None, b)):
        check_norm(hc, x, ww, bb, center, 1e-6)
    got = check_backward(hc, dy, x, None, center, 1e-6)
    xd, dyd = dev(x, dy)
    kw = dict(eps=1e-6, center=center)
    dx, dw, db = hc.hc_norm_backward(dyd, xd, None, want_dweight=False, **kw)
    assert dw is None and db is None and torch.equal(dx, got[0])
    dx, dw, db = hc.hc_norm_backward(dyd, xd, None, want_dweight=False, want_dbias=True, **kw)
    assert dw is None and torch.equal(db, got[2]) and torch.equal(dx, got[0])
    dx, dw, db = hc.hc_norm_backward(dyd, xd, None, **kw)
    assert db is None and torch.equal(dw, got[1]) and torch.equal(dx, got[0])


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("d", [64, 1000, 5120, 32776])
def test_against_differences(hc, d, center):
    """Directional differences of the 64-bit definition; the gradients' own bound along the
    direction, and 1e-5 of the terms for the difference itself."""
    x, dy, w, b = case(19, d, F32, 3)
    dx, dw, db = hc.hc_norm_backward(*dev(dy, x, w), eps=1e-5, center=center, want_dbias=True)
    a = f64(x, w, b)
    dy64 = dy.double()
    bounds = ref.norm_backward_bound(dy64, a[0], a[1], center, 1e-5, F32)
    g = torch.Generator().manual_seed(d)
    for i, (grad, bound) in enumerate(zip((dx, dw, db), bounds)):
        u = torch.randn(a[i].shape, generator=g, dtype=torch.float64)
        hi, lo = list(a), list(a)
        hi[i], lo[i] = a[i] + 1e-5 * u, a[i] - 1e-5 * u
        diff = ((ref.norm(*hi, center, 1e-5) - ref.norm(*lo, center, 1e-5)) * dy64).sum() / 2e-5
        along = grad.cpu().double() * u
        tol = (bound * u.abs()).sum() + 1e-5 * along.abs().sum()
        assert abs(float(diff - along.sum())) <= float(tol)


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("d", [128, 1000, 5120, 18440, 32776])
def test_same_bits_and_in_place(hc, d, center):
    x, dy, w, b = dev(*case(777 if d < 8192 else 50, d, BF16, 4))
    kw = dict(eps=1e-5, center=center)
    y = hc.hc_norm(x, w, b, **kw)
    got = hc.hc_norm_backward(dy, x, w, want_dbias=True, **kw)
    for a, c in zip(got, hc.hc_norm_backward(dy, x, w, want_dbias=True, **kw)):
        assert torch.equal(a, c)
    buf = dy.clone()
    again = hc.hc_norm_backward(buf, x, w, dx=buf, want_dbias=True, **kw)
    assert again[0] is buf
    for a, c in zip(got, again):
        assert torch.equal(a, c)
    buf = x.clone()
    assert hc.hc_norm(buf, w, b, y=buf, **kw) is buf and torch.equal(buf, y)
    assert torch.equal(hc.hc_norm(x.view(-1, 1, d), w, b, **kw).view_as(y), y)


@pytest.mark.parametrize("d", [40, 128, 1000, 5120, 18440, 32776])
def test_guards(hc, d):
    """What lies before and behind the outputs stays as it is."""
    rows = 13
    x, dy, w, b = dev(*case(rows, d, BF16, 5))
    for center in (False, True):
        big = [torch.full((rows * d + 128,), 7.0, dtype=BF16, device="cuda") for _ in range(2)]
        small = [torch.full((d + 64,), 7.0, device="cuda") for _ in range(2)]
        y, dx = (t[64:64 + rows * d].view(rows, d) for t in big)
        dw, db = (t[32:32 + d] for t in small)
        need = hc.hc_norm_backward_bytes(rows, d)
        ws = torch.full((need + 512,), 5, dtype=torch.uint8, device="cuda")
        assert ws.data_ptr() % 256 == 0
        hc.hc_norm(x, w, b, center=center, y=y)
        hc.hc_norm_backward(dy, x, w, center=center, dx=dx, dweight=dw, dbias=db,
                            workspace=ws[256:256 + need])
        for t, n, k in [(t, rows * d, 64) for t in big] + [(t, d, 32) for t in small]:
            assert bool((t[:k] == 7).all()) and bool((t[k + n:] == 7).all())
        assert bool((ws[:256] == 5).all()) and bool((ws[256 + need:] == 5).all())
        assert torch.equal(y, hc.hc_norm(x, w, b, center=center))


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("d", [128, 1000, 5120, 18440, 32776])
def test_bad_rows_stay_alone(hc, d, center):
    """NaN, infinities and zeros spoil their own row's outputs and no other's."""
    x, dy, w, b = case(40, d, BF16, 6)
    x[3, 5] = float("nan")
    x[7, d - 1] = float("inf")
    x[11] = 0.0
    x[12] = 2.5
    dy[17, 2] = float("nan")
    y = hc.hc_norm(*dev(x, w, b), eps=1e-5, center=center).cpu()
    dx, dw, db = (t.cpu() for t in hc.hc_norm_backward(*dev(dy, x, w), eps=1e-5, center=center,
                                                       want_dbias=True))
    good = [i for i in range(40) if i not in (3, 7, 17)]
    a = f64(x[good], w, b)
    within(y[good], ref.norm(*a, center, 1e-5), ref.norm_bound(*a, center, 1e-5, BF16), "y")
    g = f64(dy[good], x[good], w)
    want, bound = ref.norm_backward(*g, center, 1e-5), ref.norm_backward_bound(*g, center, 1e-5,
                                                                               BF16)
    within(dx[good], want[0], bound[0], "dx")
    assert torch.isnan(y[3]).all() and torch.isnan(dx[3]).all() and torch.isnan(dx[17]).all()
    assert torch.isnan(y[7]).any()
    if center:
        # a row of one number: its mean is that number, up to its sum's rounding
        off = ref.chain(d) * ref.U32 * 2.5 / 1e-5 ** 0.5
        assert torch.all((y[12].double() - b.double()).abs() <=
                         off * w.double().abs() + 2.0 ** -7 * b.double().abs())
    assert torch.isnan(dw).all()            # row 3 has NaN in every h
    assert torch.isnan(db[2]) and not torch.isnan(db[:2]).any() and not torch.isnan(db[3:]).any()


def test_extremes(hc):
    """The ends of the types: squares that leave binary32 give r = 0, small rows keep their r."""
    x = torch.zeros(4, 1000)
    x[0], x[1], x[2], x[3] = 1e30, 1e-15, 3.0, 1e-3
    x = x.to(BF16)
    y = hc.hc_norm(x.cuda(), eps=1e-20).cpu()
    assert torch.equal(y[0], torch.zeros(1000, dtype=BF16))
    a = f64(x[1:], None, None)
    within(y[1:], ref.norm(*a, False, 1e-20), ref.norm_bound(*a, False, 1e-20, BF16), "y")
    # a mean far above the deviation, in fp32
    g = torch.Generator().manual_seed(2)
    far = (1000.0 + torch.randn(3, 5120, generator=g))
    check_norm(hc, far, None, None, True, 1e-5)


@pytest.mark.parametrize("d", [64, 1000, 5120, 18440, 32776])
def test_squares_out_of_range(hc, d):
    """Rows whose squares leave binary32 have r = 0: y is the bias, dx is zero, and the row adds
    nothing to the weight's gradient.  The rows beside them are as they would be."""
    x, dy, w, b = case(12, d, BF16, 12)
    big = [1, 2, 5, 8]
    x[1], x[2] = 1e30, torch.linspace(-3e25, 2e25, d).to(BF16)
    x[5, 3], x[8, -1] = 1e33, -1e33
    rest = [i for i in range(12) if i not in big]
    for center in (False, True):
        y = hc.hc_norm(*dev(x, w, b), eps=1e-5, center=center).cpu()
        assert torch.equal(y[big], b.to(BF16).expand(4, d))
        dx, dw, db = (t.cpu() for t in hc.hc_norm_backward(*dev(dy, x, w), eps=1e-5, center=center,
                                                           want_dbias=True))
        # row 1 is one number: about its mean it has no squares, and its gradient is its own
        assert not dx[big[1:] if center else big].any()
        a, g = f64(x[rest], w, b), f64(dy[rest], x[rest], w)
        within(y[rest], ref.norm(*a, center, 1e-5), ref.norm_bound(*a, center, 1e-5, BF16), "y")
        want = ref.norm_backward(*g, center, 1e-5)
        bound = ref.norm_backward_bound(*g, center, 1e-5, BF16)
        within(dx[rest], want[0], bound[0], "dx")
        within(dw, want[1], bound[1], "dweight")
        all_dy = dy.double()
        within(db, all_dy.sum(0), bound[2] + 32 * ref.U32 * all_dy.abs().sum(0), "dbias")


def test_empty_and_shapes(hc):
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    assert hc.hc_norm(x).shape == (0, 64)
    dw = torch.ones(64, device="cuda")
    dx, dw, db = hc.hc_norm_backward(x, x, want_dbias=True, dweight=dw)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    x, dy, w, b = dev(*case(24, 64, F16, 7))
    y = hc.hc_norm(x.view(2, 3, 4, 64), w, b)
    assert y.shape == (2, 3, 4, 64) and torch.equal(y.view(24, 64), hc.hc_norm(x, w, b))
    dx = hc.hc_norm_backward(dy.view(2, 12, 64), x.view(2, 12, 64), w)[0]
    assert dx.shape == (2, 12, 64)


@pytest.mark.parametrize("d", [8, 64, 128, 520, 1000, 1272, 1288, 5120, 16384])
def test_few_rows(hc, d):
    """The most rows that one block has alone (their sums need no workspace), and one more."""
    rows = 1
    while hc.hc_norm_backward_bytes(rows + 1, d) == 0:
        rows += 1
    for center in (False, True):
        for n in (rows, rows + 1):
            x, dy, w, b = case(n, d, BF16, 13)
            got = check_backward(hc, dy, x, w, center, 1e-5)
            xd, dyd, wd = dev(x, dy, w)
            for k in ((True, False), (False, True), (False, False)):
                out = hc.hc_norm_backward(dyd, xd, wd, eps=1e-5, center=center, want_dweight=k[0],
                                          want_dbias=k[1])
                assert torch.equal(out[0], got[0])
                for a, c, want in zip(out[1:], got[1:], k):
                    assert (a is not None) == want and (a is None or torch.equal(a, c))


@pytest.mark.parametrize("d", [64, 20480])
def test_long_tensors(hc, d):
    """More than 2^31 channels: the last rows are where 32-bit offsets would fail."""
    rows = (1 << 31) // d + 100
    x = torch.zeros(rows, d, dtype=BF16, device="cuda")
    tx, tdy, w, _ = case(3, d, BF16, 8)
    x[-3:] = tx.cuda()
    y = hc.hc_norm(x, w.cuda(), eps=1e-5)
    within(y[-3:], ref.norm(*f64(tx, w), None, False, 1e-5),
           ref.norm_bound(*f64(tx, w), None, False, 1e-5, BF16), "y")
    assert int(torch.count_nonzero(y[:-3])) == 0
    y.zero_()
    y[-3:] = tdy.cuda()
    dx, dw, db = hc.hc_norm_backward(y, x, w.cuda(), eps=1e-5, want_dbias=True, dx=y)
    a = f64(tdy, tx, w)
    want, bound = ref.norm_backward(*a, False, 1e-5), ref.norm_backward_bound(*a, False, 1e-5, BF16)
    for name, g, v, t in zip(("dx", "dweight", "dbias"), (dx[-3:], dw, db), want, bound):
        within(g, v, t, name)
    assert int(torch.count_nonzero(dx[:-3])) == 0


def test_graph_streams_and_threads(hc):
    """Captured and replayed on new values, on a stream of its own, beside a call elsewhere."""
    x, dy, w, b = dev(*case(200, 5120, BF16, 9))
    ws = [torch.empty(hc.hc_norm_backward_bytes(200, 5120), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()

    def both():
        hc.hc_norm(x, w, b, center=True, eps=1e-5, y=y)
        hc.hc_norm_backward(dy, x, w, center=True, eps=1e-5, dx=dx, dweight=dw, dbias=db,
                            workspace=ws[0])

    with torch.cuda.stream(side):
        both()
        with torch.cuda.graph(graph, stream=side):
            both()
    torch.cuda.current_stream().wait_stream(side)
    x2, dy2, _, _ = dev(*case(200, 5120, BF16, 10))
    x.copy_(x2), dy.copy_(dy2)
    graph.replay()
    want = hc.hc_norm_backward(dy2, x2, w, center=True, eps=1e-5, want_dbias=True, workspace=ws[1])
    assert torch.equal(y, hc.hc_norm(x2, w, b, center=True, eps=1e-5))
    for a, c in zip((dx, dw, db), want):
        assert torch.equal(a, c)
    # the call's own outputs and workspace on another stream
    torch.cuda.synchronize()
    got = hc.hc_norm_backward(dy2, x2, w, center=True, eps=1e-5, want_dbias=True, stream=side)
    y2 = hc.hc_norm(x2, w, b, center=True, eps=1e-5, stream=side)
    side.synchronize()
    assert torch.equal(y2, y)
    for a, c in zip(got, want):
        assert torch.equal(a, c)


def test_refusals(hc):
    x = torch.zeros(8, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        hc.hc_norm(x.t().contiguous().t())
    with pytest.raises(ValueError):
        hc.hc_norm(x, w[:32])
    with pytest.raises(TypeError):
        hc.hc_norm(x, w.to(BF16))
    with pytest.raises(ValueError):
        hc.hc_norm(x, w.cpu())
    with pytest.raises(TypeError):
        hc.hc_norm(x, y=torch.empty(8, 64, device="cuda"))
    with pytest.raises(hc.HcError, match="MISALIGNED"):
        hc.hc_norm(torch.zeros(8, 12, dtype=BF16, device="cuda"))
    with pytest.raises(hc.HcError, match="INVALID"):
        hc.hc_norm(x, eps=-1.0)
    with pytest.raises(TypeError):
        hc.hc_norm_backward(x.float(), x)
    with pytest.raises(ValueError):
        hc.hc_norm_backward(x[:4], x)
    many = torch.zeros(800, 1000, dtype=BF16, device="cuda")
    with pytest.raises(hc.HcError, match="INVALID"):
        hc.hc_norm_backward(many, many, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [8, 40, 128, 1000, 5120, 18440, 32776])
def test_layer_norm_of_rows_that_start_apart(hc, d, dtype):
    """Rows whose first channels say nothing of their mean, beside ordinary ones: outliers in front,
    a far mean behind zeros, one number in all channels but the last."""
    x, dy, w, b = case(41, d, dtype, 11)
    x[1, 0], x[2, :4] = 3000.0, -2000.0
    x[5] = 700.0 + x[5]
    x[5, :8] = 0.0
    x[9], x[9, -1] = 2.5, 2.0
    x[13] = -1.0
    x[20] += 500.0
    check_norm(hc, x, w, b, True, 1e-5)
    check_backward(hc, dy, x, w, True, 1e-5)
