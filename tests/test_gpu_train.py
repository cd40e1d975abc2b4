"""The training operators against their 64-bit forms (GPU)."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import train_reference as ref

pytestmark = pytest.mark.gpu
U32, UBF = ref.U32, ref.UBF
NORM_EPS = 1e-20


@pytest.fixture(scope="module")
def hc():
    import sinkhorn_mixing_gb300 as lib
    lib.lib()
    yield lib
    assert lib.hc_device_error(clear=True) == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bf16(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def kept_of(hc, t, k8):
    return hc.hc_checkpoint(t) if k8 else t


# ------------------------------------------------------- rows kept in 8 bits

SHAPES = [(1, 8), (3, 24), (5, 32), (7, 40), (33, 64), (2, 1000), (130, 96), (1, 5120), (17, 5120),
          (4099, 72)]


def check_kept(hc, x):
    codes, scales = hc.hc_checkpoint(x)
    b = bits(x).reshape(-1, x.shape[-1])
    want_c, want_s = ref.checkpoint(b)
    assert np.array_equal(scales.cpu().numpy().reshape(want_s.shape), want_s)
    assert np.array_equal(codes.cpu().view(torch.uint8).numpy().reshape(want_c.shape), want_c)
    back = hc.hc_restore(codes, scales)
    v = ref.values((codes, scales))
    assert torch.equal(torch.isnan(back.cpu()), torch.isnan(v))
    ok = ~torch.isnan(v)
    assert torch.equal(back.cpu().double()[ok], v[ok])


@pytest.mark.parametrize("rows,d", SHAPES)
def test_checkpoint_restore(hc, rows, d):
    g = gen(rows * 7 + d)
    x = torch.randn(rows, d, generator=g) * torch.exp(4 * torch.randn(rows, 1, generator=g))
    x[0, 0] = 0.0
    check_kept(hc, x.to(torch.bfloat16).cuda())


def test_checkpoint_every_number(hc):
    b = np.arange(65536, dtype=np.uint16)
    for order in (b, np.random.RandomState(0).permutation(b)):
        x = torch.from_numpy(order.view(np.int16).copy()).view(torch.bfloat16)
        check_kept(hc, x.reshape(-1, 64).cuda())
        check_kept(hc, x[:65520].reshape(-1, 40).cuda())


def test_checkpoint_special_blocks(hc):
    x = torch.zeros(8, 64)
    x[1, 3] = float("inf")
    x[2] = float("nan")
    x[3, 5], x[3, 7] = float("-inf"), 2.0 ** -133
    x[4] = -0.0
    x[5] = 3.38e38
    x[6, :32] = torch.linspace(-448, 448, 32)
    x[7, 0] = 449.0
    check_kept(hc, x.to(torch.bfloat16).cuda())


def test_checkpoint_shapes_and_empty(hc):
    x = bf16((2, 3, 4, 72), gen(1)).cuda()
    codes, scales = hc.hc_checkpoint(x)
    assert codes.shape == x.shape and scales.shape == (2, 3, 4, 3)
    assert hc.hc_restore(codes, scales).shape == x.shape
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    c, s = hc.hc_checkpoint(e)
    assert c.shape == (0, 4, 64) and hc.hc_restore(c, s).shape == (0, 4, 64)


def test_scales_at_any_address(hc):
    # a batch cut by tokens: 12 scale bytes a token, so the cut's scales are not aligned
    g = gen(4)
    x = bf16((40, 4, 72), g).cuda()
    codes, scales = hc.hc_checkpoint(x)
    cut = (codes[1:].contiguous(), scales[1:])
    assert scales[1:].data_ptr() % 16 == 12
    assert torch.equal(hc.hc_restore(*cut), hc.hc_restore(codes, scales)[1:])
    pre = torch.rand(40, 4, generator=g).cuda()
    assert torch.equal(hc.hc_pre_restore(*cut, pre[1:].contiguous()),
                       hc.hc_pre_restore(codes, scales, pre)[1:])
    out = torch.full((500,), 7, dtype=torch.uint8, device="cuda")
    _, s2 = hc.hc_checkpoint(x, scales=out[5:485].view(40, 4, 3))
    assert torch.equal(s2, scales) and bool((out[:5] == 7).all()) and bool((out[485:] == 7).all())
    c = pre_case(hc, 40, 4, 72, True)
    d = dict(c, x=(c["x"][0], torch.cat([c["x"][1].view(-1)[:1], c["x"][1].view(-1)])[1:]
                   .view(40, 4, 3)))
    assert d["x"][1].data_ptr() % 16 == 1
    for a, b in zip(run_pre(hc, d), run_pre(hc, c)):
        assert torch.equal(a, b)


def test_checkpoint_long_tensor(hc):
    # more than 2^31 channels: the last rows are where 32-bit offsets would fail
    n, d = 110_000, 20480
    x = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    tail = bf16((3, d), gen(9)).cuda()
    x[-3:] = tail
    codes, scales = hc.hc_checkpoint(x)
    want_c, want_s = ref.checkpoint(bits(tail))
    assert np.array_equal(codes[-3:].cpu().view(torch.uint8).numpy(), want_c)
    assert np.array_equal(scales[-3:].cpu().numpy(), want_s)
    x.fill_(1.0)
    hc.hc_restore(codes, scales, x=x)
    assert torch.equal(x[-3:].cpu().double(), ref.values((codes[-3:], scales[-3:])))
    assert int(torch.count_nonzero(x[:-3])) == 0
    pre = torch.rand(n // 4, 4, generator=gen(2)).cuda()
    y = hc.hc_pre_restore(codes.view(-1, 4, d), scales.view(n // 4, 4, -1), pre)
    w = torch.einsum("j,jc->c", pre[-1].cpu().double(),
                     ref.values((codes[-4:], scales[-4:])))
    assert torch.all((y[-1].cpu().double() - w).abs() <= UBF * w.abs() + 1e-6)


@pytest.mark.parametrize("copies", [4, 8])
@pytest.mark.parametrize("n,d", [(1, 8), (3, 40), (5, 72), (257, 64), (2, 1000), (31, 5120)])
def test_pre_restore(hc, copies, n, d):
    g = gen(n + d + copies)
    x = bf16((n, copies, d), g, 3.0).cuda()
    pre = torch.rand(n, copies, generator=g).cuda()
    codes, scales = hc.hc_checkpoint(x)
    y = hc.hc_pre_restore(codes, scales, pre)
    v, p = ref.values((codes, scales)), pre.cpu().double()
    want = torch.einsum("nj,njc->nc", p, v)
    mag = torch.einsum("nj,njc->nc", p.abs(), v.abs())
    assert torch.all((y.cpu().double() - want).abs() <= UBF * want.abs() + 2 * copies * U32 * mag)
    # the collapse of the restored stream, bit for bit
    assert torch.equal(y, hc.hc_pre(hc.hc_restore(codes, scales), pre))


@pytest.mark.parametrize("copies", [4, 8])
@pytest.mark.parametrize("n,d", [(1, 8), (3, 40), (257, 64), (2, 1000), (31, 5120)])
@pytest.mark.parametrize("in_place", [False, True])
def test_post_checkpoint(hc, copies, n, d, in_place):
    g = gen(n * 3 + d + copies)
    res, out = bf16((n, copies, d), g).cuda(), bf16((n, d), g).cuda()
    post = torch.rand(n, copies, generator=g).cuda()
    comb = torch.rand(n, copies, copies, generator=g).cuda()
    want = hc.hc_post(out, res, post, comb)
    wc, ws = hc.hc_checkpoint(want)
    y, codes, scales = hc.hc_post_checkpoint(out, res, post, comb, y=res if in_place else None)
    assert torch.equal(y, want)
    assert torch.equal(codes.view(torch.uint8), wc.view(torch.uint8))
    assert torch.equal(scales, ws)


# --------------------------------------------------------------- hc_post's

def post_case(hc, n, copies, d, r8, o8, seed=0):
    g = gen(n * 5 + d + copies + seed)
    dy = bf16((n, copies, d), g, 2.0 ** -6).cuda()
    out = kept_of(hc, bf16((n, d), g).cuda(), o8)
    res = kept_of(hc, bf16((n, copies, d), g, 2.0).cuda(), r8)
    post = (2 * torch.rand(n, copies, generator=g)).cuda()
    comb = torch.rand(n, copies, copies, generator=g).cuda()
    return dy, out, res, post, comb


def check_post(got, dy, out, res, post, comb):
    copies, d = dy.shape[-2:]
    grads, mags = ref.post_backward(dy.cpu().double(), ref.values(out), ref.values(res),
                                    post.cpu().double(), comb.cpu().double())
    # a chain of at most d/32 + 8 products per lane, 5 steps over the lanes, 8 over warps
    k = d / 32 + 8 + 5 + 8
    for name, t, want, mag in zip(("dout", "dpost", "dcomb", "dresidual"), got, grads, mags):
        if t is None:
            continue
        t = t.cpu().double()
        if name in ("dpost", "dcomb"):
            tol = (k + 1) * U32 * mag
        else:
            tol = UBF * want.abs() + (copies + 1) * U32 * mag
        bad = (t - want).abs() > tol
        assert not bad.any(), (name, int(bad.sum()), float((t - want).abs().max()))


@pytest.mark.parametrize("copies", [4, 8])
@pytest.mark.parametrize("n,d", [(1, 8), (2, 24), (9, 40), (130, 64), (3, 1000), (7, 5120),
                                 (2500, 264)])
@pytest.mark.parametrize("r8,o8,dres", [(True, True, False), (False, False, True),
                                        (True, False, True), (False, True, False)])
def test_post_backward(hc, copies, n, d, r8, o8, dres):
    args = post_case(hc, n, copies, d, r8, o8)
    got = hc.hc_post_backward(*args, want_dresidual=dres)
    assert (got[3] is not None) == dres
    check_post(got, *args)


@pytest.mark.parametrize("copies", [4, 8])
def test_post_backward_in_place(hc, copies):
    dy, out, res, post, comb = post_case(hc, 37, copies, 200, True, True)
    want = hc.hc_post_backward(dy, out, res, post, comb, want_dresidual=True)
    buf = dy.clone()
    got = hc.hc_post_backward(buf, out, res, post, comb, dresidual=buf)
    assert got[3] is buf
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_post_backward_long_tensor(hc):
    n, copies, d = 27_000, 4, 20480
    dy = torch.zeros(n, copies, d, dtype=torch.bfloat16, device="cuda")
    res = torch.zeros_like(dy)
    out = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    args = post_case(hc, 2, copies, d, False, False)
    dy[-2:], out[-2:], res[-2:] = args[0], args[1], args[2]
    post, comb = torch.ones(n, copies, device="cuda"), torch.ones(n, copies, copies, device="cuda")
    post[-2:], comb[-2:] = args[3], args[4]
    got = hc.hc_post_backward(dy, out, res, post, comb, dresidual=dy)
    assert int(torch.count_nonzero(got[2][:-2])) == 0
    check_post([t[-2:] for t in got], *args)


# ---------------------------------------------------------- hc_mixes_pre's

def pre_case(hc, n, copies, d, k8, dstream=True, scale_range=1.5, base_std=1.0, seed=0):
    g = gen(n * 11 + d + copies + seed)
    F, mix = copies * d, (2 + copies) * copies
    x = torch.randn(n, copies, d, generator=g) * torch.exp(torch.randn(n, 1, 1, generator=g))
    c = dict(dy=bf16((n, d), g, 2.0 ** -6), x=x.to(torch.bfloat16),
             w=torch.randn(mix, F, generator=g) * F ** -0.5,
             scale=0.5 + scale_range * torch.rand(3, generator=g),
             base=base_std * torch.randn(mix, generator=g),
             dpost=0.1 * torch.randn(n, copies, generator=g),
             dcomb=0.1 * torch.randn(n, copies, copies, generator=g),
             dstream=bf16((n, copies, d), g, 2.0 ** -6) if dstream else None)
    c = {k: v if v is None else v.cuda() for k, v in c.items()}
    c["x"] = kept_of(hc, c["x"], k8)
    m = ref.mixes(ref.values(c["x"]), c["w"].cpu().double(), NORM_EPS)
    c["mixes"] = m.float().cuda()
    return c


def run_pre(hc, c, iters=20, norm_eps=NORM_EPS, **more):
    return hc.hc_mixes_pre_backward(c["dy"], c["x"], c["mixes"], c["w"], c["scale"], c["base"],
                                    c["dpost"], c["dcomb"], dstream=c["dstream"],
                                    sinkhorn_iters=iters, norm_eps=norm_eps, **more)


def check_pre(got, c, iters=20, norm_eps=NORM_EPS):
    f64 = lambda t: None if t is None else t.detach().cpu().double()  # noqa: E731
    x = ref.values(c["x"])
    n, copies, d = x.shape
    (dx, dw, dscale, dbase), t = ref.mixes_pre_backward(
        f64(c["dy"]), x, f64(c["mixes"]), f64(c["w"]), f64(c["scale"]), f64(c["base"]),
        f64(c["dpost"]), f64(c["dcomb"]), f64(c["dstream"]), iters, 1e-6, norm_eps)
    gx, gw, gs, gb = (f64(v) for v in got)
    # sums over channels (dpre, the mean square): see check_post; over a token's mix numbers; and
    # the split
    split = ref.split_tolerance(iters)
    sums = (d / 32 + 21 + t["du"].shape[1]) * U32
    # an error of du, relative to the largest of the token's: dpre's terms may cancel
    du = t["du"]
    dpre_mag = (f64(c["dy"]).abs()[:, None] * x.abs()).sum(2)
    r = (x.flatten(1).square().mean(1, keepdim=True) + norm_eps) ** -0.5
    du_err = (split * du.norm(dim=1) + (sums * dpre_mag.amax(1) * r[:, 0]) *
              float(c["scale"].abs().max()))                       # [n]
    wsum = f64(c["w"]).abs().sum(0).view(copies, d)
    # dx: its rounding to bf16; du's error through W; the product's factors in 11 bits (half a
    # step of 2^-11 each); the other terms in binary32, q among them
    tol = (UBF * dx.abs() + du_err[:, None, None] * wsum + 2.0 ** -10 * t["proj"] +
           (split + (16 + copies) * U32) * t["rest"] + sums * t["rest"])
    bad = (gx - dx).abs() > tol
    assert not bad.any(), ("dx", int(bad.sum()), float(((gx - dx).abs() - tol).max()))
    # dw: du's error; its three bf16 parts (2^-24 left); a chain over the tokens
    dw_tol = ((du_err[:, None] * x.flatten(1).abs()).sum(0)[None] +
              (n ** 0.5 * 4 + 32) * U32 * t["dw"])
    bad = (gw - dw).abs() > dw_tol
    assert not bad.any(), ("dw", int(bad.sum()), float(((gw - dw).abs() - dw_tol).max()))
    # dbase, dscale: the same errors of dz, before r and the scales
    dz_err = (du_err / (r[:, 0] * float(c["scale"].abs().min()))).sum() + \
        (n ** 0.5 * 4 + 32) * U32 * (du.abs() / r).sum() / float(c["scale"].abs().min())
    assert torch.all((gb - dbase).abs() <= dz_err), ("dbase", float((gb - dbase).abs().max()))
    m = f64(c["mixes"]).abs()
    assert torch.all((gs - dscale).abs() <= dz_err * m.max() * m.shape[1]), "dscale"


PRE = [(1, 8), (2, 24), (7, 32), (9, 40), (17, 64), (130, 72), (33, 1000), (16, 1024), (5, 5120),
       (700, 264)]


@pytest.mark.parametrize("copies", [4, 8])
@pytest.mark.parametrize("n,d", PRE)
@pytest.mark.parametrize("k8", [True, False])
def test_mixes_pre_backward(hc, copies, n, d, k8):
    c = pre_case(hc, n, copies, d, k8)
    check_pre(run_pre(hc, c), c)


@pytest.mark.parametrize("n,d", [(2, 64), (63, 80), (64, 96), (65, 128), (700, 144), (1100, 192),
                                 (3000, 5120), (128, 64), (129, 80), (190, 96), (193, 1040),
                                 (1025, 264)])
@pytest.mark.parametrize("k8", [True, False])
def test_mixes_pre_backward_streamed(hc, monkeypatch, n, d, k8):
    # shapes that the TMA kernel takes, and the general path on the same inputs
    c = pre_case(hc, n, 4, d, k8)
    got = run_pre(hc, c)
    check_pre(got, c)
    monkeypatch.setenv("HCMIX_PATH", "general")
    other = run_pre(hc, c)
    check_pre(other, c)
    assert torch.equal(got[2], other[2]) and torch.equal(got[3], other[3])


@pytest.mark.parametrize("copies", [4, 8])
@pytest.mark.parametrize("iters", [1, 2, 50, 256])
def test_mixes_pre_backward_iters(hc, copies, iters):
    c = pre_case(hc, 21, copies, 96, True, seed=iters)
    check_pre(run_pre(hc, c, iters=iters), c, iters=iters)


@pytest.mark.parametrize("copies", [4, 8])
def test_mixes_pre_backward_no_stream_and_in_place(hc, copies):
    c = pre_case(hc, 50, copies, 328, True)
    want = run_pre(hc, c)
    buf = c["dstream"].clone()
    got = run_pre(hc, dict(c, dstream=buf), dx=buf)
    assert got[0] is buf
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    none = dict(c, dstream=None)
    zero = dict(c, dstream=torch.zeros_like(c["dstream"]))
    for a, b in zip(run_pre(hc, none), run_pre(hc, zero)):
        assert torch.equal(a, b)
    check_pre(run_pre(hc, none), none)


@pytest.mark.parametrize("copies", [4, 8])
def test_mixes_pre_backward_zero_token(hc, copies):
    # a padded token: no stream, no gradient; r is 1 / sqrt(norm_eps)
    c = pre_case(hc, 12, copies, 64, False)
    for k in ("x", "dy", "dstream", "dpost", "dcomb", "mixes"):
        c[k][5] = 0
    got = run_pre(hc, c, norm_eps=1e-6)
    assert int(torch.count_nonzero(got[0][5])) == 0
    keep = [i for i in range(12) if i != 5]
    less = {k: (v[keep].contiguous() if k in ("x", "dy", "dstream", "dpost", "dcomb", "mixes")
                else v) for k, v in c.items()}
    few = run_pre(hc, less, norm_eps=1e-6)
    assert torch.equal(got[0][keep], few[0])
    # the sums differ by their order over the tokens alone
    for a, b in zip(got[1:], few[1:]):
        assert torch.allclose(a, b, rtol=1e-5, atol=1e-5 * float(b.abs().max()))


def test_mixes_pre_backward_nan_stays_in_its_token(hc):
    c = pre_case(hc, 40, 4, 264, False)
    want = run_pre(hc, c)[0]
    c["dy"][17, 5] = float("nan")
    got = run_pre(hc, c)[0]
    keep = [i for i in range(40) if i != 17]
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[17]).any()


@pytest.mark.parametrize("copies", [4, 8])
def test_mixes_pre_backward_against_differences(hc, copies):
    # the loss along random directions, by differences of the 64-bit forward pass
    n, d = 6, 64
    c = pre_case(hc, n, copies, d, False, dstream=False)
    got = [t.cpu().double() for t in run_pre(hc, c)]
    f64 = lambda t: t.detach().cpu().double()  # noqa: E731
    at = [f64(c["x"]), f64(c["w"]), f64(c["scale"]), f64(c["base"])]

    def loss(x, w, scale, base):
        y, _, po, co, _ = ref.mixes_pre(x, w, scale, base, 20, 1e-6, NORM_EPS)
        return ((y * f64(c["dy"])).sum() + (po * f64(c["dpost"])).sum() +
                (co * f64(c["dcomb"])).sum())

    g = gen(5)
    for i in range(4):
        v = torch.randn(at[i].shape, generator=g, dtype=torch.float64)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + 1e-5 * v, at[i] - 1e-5 * v
        num = (loss(*up) - loss(*down)) / 2e-5
        mag = (got[i] * v).abs().sum()
        # dx is rounded to bf16, and its product term to 11 bits; the sums are binary32
        tol = (UBF + 2.0 ** -9 if i == 0 else ref.split_tolerance(20) * 4) * mag
        assert abs(num - (got[i] * v).sum()) <= tol + 1e-6 * mag, i


def test_mixes_pre_backward_no_tokens(hc):
    z = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    got = hc.hc_mixes_pre_backward(
        z(0, 64, dt=torch.bfloat16), z(0, 4, 64, dt=torch.bfloat16), z(0, 24), z(24, 256), z(3),
        z(24), z(0, 4), z(0, 4, 4), dw_mix=torch.ones(24, 256, device="cuda"))
    assert got[0].shape == (0, 4, 64)
    for t in got[1:]:
        assert int(torch.count_nonzero(t)) == 0


# ------------------------------------------------- streams, graphs, guards

def test_same_bits_every_time(hc):
    for copies in (4, 8):
        c = pre_case(hc, 1500, copies, 136, True)
        first = run_pre(hc, c)
        for _ in range(3):
            for a, b in zip(run_pre(hc, c), first):
                assert torch.equal(a, b)


@pytest.mark.parametrize("k8", [True, False])
def test_two_threads_with_different_steps(hc, k8):
    # the steps set the coefficients kernel's shared memory: 131 KB and 77 KB here
    c = pre_case(hc, 9, 8, 64, k8)
    steps = (256, 150)
    want = [run_pre(hc, c, iters=i) for i in steps]
    torch.cuda.synchronize()
    failed = []

    def calls(which):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(300):
                    got = run_pre(hc, c, iters=steps[which])
                s.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want[which]))
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_outputs_for_another_stream(hc):
    # a tensor freed while the current stream has still to read it is not an output of another
    # stream's call: same size, so that the allocator would hand the block out at once
    codes, scales = hc.hc_checkpoint(torch.full((4096, 256), 3.0, dtype=torch.bfloat16,
                                                device="cuda"))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    block = torch.full((4096, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    at = block.data_ptr()
    kept = torch.empty_like(block)
    torch.cuda._sleep(50_000_000)
    kept.copy_(block)
    del block
    got = hc.hc_restore(codes, scales, stream=s)
    assert got.data_ptr() != at
    # and the other way round: read on the current stream, freed, made again for s
    s.synchronize()
    torch.cuda._sleep(50_000_000)
    again = got.clone()
    at = got.data_ptr()
    del got
    assert hc.hc_restore(codes, scales, stream=s).data_ptr() != at
    torch.cuda.synchronize()
    assert bool((kept == 5.0).all()) and bool((again == 3.0).all())


def test_on_another_stream_and_in_a_graph(hc):
    c = pre_case(hc, 300, 4, 512, True)
    p = post_case(hc, 300, 4, 512, True, True)
    want = run_pre(hc, c) + hc.hc_post_backward(*p, want_dresidual=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = run_pre(hc, c, stream=s) + hc.hc_post_backward(*p, want_dresidual=True, stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # two captured graphs, each with a workspace of its own, replayed in turn and at once
    with torch.cuda.stream(s):
        run_pre(hc, c)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run_pre(hc, c) + hc.hc_post_backward(*p, want_dresidual=True))
        graphs.append(g)
    s2 = torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
        torch.cuda.synchronize()
        for o in outs:
            for a, b in zip(o, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("copies", [4, 8])
@pytest.mark.parametrize("n,d,k8", [(1, 8, True), (13, 40, False), (37, 264, True),
                                    (130, 1032, False)])
def test_nothing_outside_the_outputs(hc, copies, n, d, k8):
    guard = 64

    def framed(shape, dtype):
        count = int(np.prod(shape))
        item = torch.empty((), dtype=dtype).element_size()
        raw = torch.full((count * item + 2 * guard * 16,), 0xA5, dtype=torch.uint8, device="cuda")
        return raw, raw[guard * 16:guard * 16 + count * item].view(dtype).view(shape)

    c = pre_case(hc, n, copies, d, k8)
    mix = (2 + copies) * copies
    wbytes = hc.hc_mixes_pre_backward_bytes(n, copies, d)
    ws = torch.full((wbytes + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    outs = dict(dx=((n, copies, d), torch.bfloat16), dw_mix=((mix, copies * d), torch.float32),
                dscale=((3,), torch.float32), dbase=((mix,), torch.float32))
    made = {k: framed(*v) for k, v in outs.items()}
    run_pre(hc, c, workspace=ws[:wbytes], **{k: v[1] for k, v in made.items()})
    p = post_case(hc, n, copies, d, k8, k8)
    outs = dict(dout=((n, d), torch.bfloat16), dpost=((n, copies), torch.float32),
                dcomb=((n, copies, copies), torch.float32),
                dresidual=((n, copies, d), torch.bfloat16))
    more = {k: framed(*v) for k, v in outs.items()}
    hc.hc_post_backward(*p, **{k: v[1] for k, v in more.items()})
    nblk = -(-d // 32)
    kept = dict(codes=framed((n, copies, d), torch.float8_e4m3fn),
                scales=framed((n, copies, nblk), torch.uint8))
    hc.hc_checkpoint(p[0], **{k: v[1] for k, v in kept.items()})
    back = dict(x=framed((n, copies, d), torch.bfloat16))
    hc.hc_restore(kept["codes"][1], kept["scales"][1], x=back["x"][1])
    low = dict(y=framed((n, d), torch.bfloat16))
    hc.hc_pre_restore(kept["codes"][1], kept["scales"][1], p[3], y=low["y"][1])
    full = dict(y=framed((n, copies, d), torch.bfloat16),
                codes=framed((n, copies, d), torch.float8_e4m3fn),
                scales=framed((n, copies, nblk), torch.uint8))
    hc.hc_post_checkpoint(bf16((n, d), gen(1)).cuda(), p[0], p[3], p[4],
                          **{k: v[1] for k, v in full.items()})
    torch.cuda.synchronize()
    assert bool((ws[wbytes:] == 0xA5).all())
    for group in (made, more, kept, back, low, full):
        for k, (raw, _) in group.items():
            assert bool((raw[:guard * 16] == 0xA5).all()) and \
                bool((raw[-guard * 16:] == 0xA5).all()), k


def test_refusals(hc):
    c = pre_case(hc, 6, 4, 64, True)
    ok = dict(c)
    for key, bad, err in (
            ("w", c["w"][:, :-4].contiguous(), ValueError),
            ("mixes", c["mixes"][:5].contiguous(), ValueError),
            ("dy", c["dy"][:5].contiguous(), ValueError),
            ("dy", c["dy"].float(), TypeError),
            ("dpost", c["dpost"].cpu(), ValueError),
            ("dstream", c["dstream"].transpose(1, 2), ValueError),
            ("x", (c["x"][0], c["x"][1][..., :1].contiguous()), ValueError),
            ("x", (c["x"][0],), TypeError),
            ("base", c["base"][:20].contiguous(), ValueError)):
        with pytest.raises(err):
            run_pre(hc, dict(ok, **{key: bad}))
    with pytest.raises(hc.HcError):
        run_pre(hc, c, iters=257)
    with pytest.raises(hc.HcError):
        run_pre(hc, c, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(hc.HcError):
        run_pre(hc, c, dw_mix=c["w"])                 # an output on an input
    codes, scales = c["x"]
    with pytest.raises(ValueError):
        hc.hc_restore(codes, scales[..., :1].contiguous())
    with pytest.raises(TypeError):
        hc.hc_restore(codes.view(torch.uint8), scales)
    with pytest.raises(hc.HcError):
        hc.hc_checkpoint(torch.zeros(2, 12, dtype=torch.bfloat16, device="cuda"))


# -------------------------------------------------------- a run of them all

@pytest.mark.parametrize("copies", [4, 8])
@pytest.mark.parametrize("k8", [True, False])
def test_two_sublayers_forward_and_backward(hc, copies, k8):
    """Two sublayers (y -> y A) trained for a step as a user would: the forward calls, streams
    kept at each boundary, the sublayer recomputed from them, the gradient calls; against
    automatic differentiation of the whole in 64 bits on the streams as kept."""
    n, d, mix = 96, 256, (2 + copies) * copies
    g = gen(copies + k8)
    A = [torch.randn(d, d, generator=g) * d ** -0.5 for _ in range(2)]
    P = [dict(w=torch.randn(mix, copies * d, generator=g) * (copies * d) ** -0.5,
              scale=0.5 + torch.rand(3, generator=g), base=torch.randn(mix, generator=g))
         for _ in range(2)]
    x0, top = bf16((n, copies, d), g), bf16((n, copies, d), g, 2.0 ** -6)

    # forward: one stream per boundary is kept, and the mix numbers
    x, keep = x0.cuda(), []
    ck = hc.hc_checkpoint(x) if k8 else x.clone()
    for i in range(2):
        p = {k: v.cuda() for k, v in P[i].items()}
        y, pre, post, comb, m = hc.hc_mixes_pre(x, p["w"], p["scale"], p["base"], want_mixes=True)
        out = (y.float() @ A[i].cuda()).to(torch.bfloat16)
        keep.append((ck, m, pre, post, comb, p))
        if k8:
            x, c8, s8 = hc.hc_post_checkpoint(out, x, post, comb)
            ck = (c8, s8)
        else:
            x = hc.hc_post(out, x, post, comb)
            ck = x
    # backward
    grad, got = top.cuda(), []
    for i in (1, 0):
        ck, m, pre, post, comb, p = keep[i]
        y = hc.hc_pre_restore(*ck, pre) if k8 else hc.hc_pre(ck, pre)
        out = (y.float() @ A[i].cuda()).to(torch.bfloat16)
        dout, dpost, dcomb, _ = hc.hc_post_backward(grad, out, ck, post, comb)
        dA = y.float().t() @ dout.float()
        dy = (dout.float() @ A[i].cuda().t()).to(torch.bfloat16)
        grad, dw, ds, db = hc.hc_mixes_pre_backward(dy, ck, m, p["w"], p["scale"], p["base"],
                                                    dpost, dcomb, dstream=grad, dx=grad)
        got.append((dA, dw, ds, db))
    torch.cuda.synchronize()

    # the same step in 64 bits: each boundary's stream takes the value that was kept
    leaves, total = [], None
    xs = ref.values(keep[0][0]).requires_grad_()
    cur = xs
    for i in range(2):
        a = A[i].double().requires_grad_()
        w, s, b = (P[i][k].double().requires_grad_() for k in ("w", "scale", "base"))
        leaves.append((a, w, s, b))
        y, _, po, co, _ = ref.mixes_pre(cur, w, s, b, 20, 1e-6, NORM_EPS)
        nxt = ref.post(y @ a, cur, po, co)
        if i == 0:
            nxt = nxt + (ref.values(keep[1][0]) - nxt).detach()
        cur = nxt
    flat = [t for l in leaves for t in l]
    grads = torch.autograd.grad((cur * top.double()).sum(), [xs] + flat)
    # bf16 roundings along the way (y, out, dout, dy, each boundary's gradient: about ten of
    # them), and 8-bit streams' mix numbers are those of the streams before they were kept
    # (2^-4 a channel, at random over copies * d channels, through two sublayers)
    tol = 10 * UBF / 2 + (2.0 ** -4 * 4 if k8 else 0)
    assert float((grad.cpu().double() - grads[0]).norm() / grads[0].norm()) <= tol
    for i, (dA, dw, ds, db) in zip((1, 0), got):
        for t, want in zip((dA, dw, ds, db), grads[1 + 4 * i:5 + 4 * i]):
            assert float((t.cpu().double() - want).norm() / want.norm()) <= 2 * tol, i
