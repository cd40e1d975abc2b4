"""hc_mixes_pre_backward over long runs of steps, and a training step on restored streams (GPU).

A block of the kernels that make dx and dW walks over up to n / 38 tokens in steps of 16 (hc = 8) or
32, and moves dW's running sums on every 16 steps.  The shapes here give every block more than two
such moves, whatever the GPU's number of SMs (148 to 160).
"""
import pytest
import torch

import test_gpu_train as t
import train_reference as ref

pytestmark = pytest.mark.gpu
U32, UBF, NORM_EPS = ref.U32, ref.UBF, t.NORM_EPS


@pytest.fixture(scope="module")
def hc():
    import sinkhorn_mixing_gb300 as lib
    lib.lib()
    yield lib
    assert lib.hc_device_error(clear=True) == 0


# steps a block walks over without a break: 48 and 39 at hc = 8; 38 at hc = 4
@pytest.mark.parametrize("copies,n,d", [(8, 24571, 264), (8, 6144, 1000), (4, 24011, 1000)])
@pytest.mark.parametrize("k8", [True, False])
def test_long_runs(hc, monkeypatch, copies, n, d, k8):
    monkeypatch.setenv("HCMIX_PATH", "general")
    c = t.pre_case(hc, n, copies, d, k8)
    t.check_pre(t.run_pre(hc, c), c)


@pytest.mark.parametrize("copies,k8,path", [(4, True, "auto"), (4, False, "auto"),
                                            (4, False, "general"), (8, True, "auto"),
                                            (8, False, "auto")])
def test_sums_that_all_have_one_sign(hc, monkeypatch, copies, k8, path):
    """dW where nothing cancels: x and dpost are positive, dy and dcomb are zero, so that du of
    post's mix numbers is positive and all others are zero.  About 1,000 steps a block.

    The tensor core rounds a running sum toward zero, so in a sum of positive terms its errors all
    have one sign.  A step adds 2 (hc = 4) or 3 (hc = 8: three parts in turn) products of 16 tokens,
    each at most 2 units of 2^-23 of the sum off (the products' alignment, the sum's end); 16 steps
    until the sums move on; then at most 1,100 / 16 moves and 200 partial sums, rounded to nearest
    (2^-24 each); du itself about 16 roundings and the mean square's sum (see check_pre).  Sums that
    never moved on would be 2,000 or 3,000 such additions off, each by half a unit of 2^-23.5 on
    average while the sum grows: 4e-5 to 6e-5, well above the bound."""
    if path == "general":
        monkeypatch.setenv("HCMIX_PATH", "general")
    mix = (2 + copies) * copies
    # four slices of channels, walked over by teams of four blocks
    tokens, d = (32, 512) if path == "general" else (32 if copies == 4 else 16, 256)
    n = 1000 * tokens * 38 + 7
    g = torch.Generator(device="cuda").manual_seed(copies)
    F = copies * d
    x = torch.empty(n, copies, d, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g).abs_()
    kept = hc.hc_checkpoint(x) if k8 else x
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    scale, base = torch.full((3,), 1.25, device="cuda"), rand(mix) - 0.5
    mixes, dpost = 2 * rand(n, mix) - 1, 0.5 + rand(n, copies)
    w = (rand(mix, F) - 0.5) * F ** -0.5
    zero = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    _, dw, _, dbase = hc.hc_mixes_pre_backward(
        zero, kept, mixes, w, scale, base, dpost, torch.zeros(n, copies, copies, device="cuda"),
        norm_eps=NORM_EPS)

    want, want_base = torch.zeros(copies, F, dtype=torch.float64, device="cuda"), 0.0
    for i in range(0, n, 1 << 15):
        if k8:
            f = torch.exp2(kept[1][i:i + (1 << 15)].double() - 127.0).repeat_interleave(32, -1)
            v = kept[0][i:i + (1 << 15)].float().double() * f
        else:
            v = x[i:i + (1 << 15)].double()
        v = v.flatten(1)
        r = (v.square().mean(1, keepdim=True) + NORM_EPS) ** -0.5
        z = mixes[i:i + (1 << 15), copies:2 * copies].double() * 1.25 + \
            base[copies:2 * copies].double()
        s = torch.sigmoid(z)
        dz = 2.0 * dpost[i:i + (1 << 15)].double() * s * (1 - s)
        want += (dz * 1.25 * r).t() @ v
        want_base = want_base + dz.sum(0)
    post = dw[copies:2 * copies].double()
    chunk = 16 * (2 if copies == 4 else 3) * 2 * 2.0 ** -23
    bound = chunk + (1100 / 16 + 200) * U32 + (16 + F / 8 / 32 + 21) * U32
    err = ((post - want) / want).abs()
    assert float(err.max()) <= bound, (float(err.max()), bound)
    others = [i for i in range(mix) if not copies <= i < 2 * copies]
    assert int(torch.count_nonzero(dw[others])) == 0
    # a lane adds up n / 2,400 tokens at least, a few thousand at most
    assert torch.all((dbase[copies:2 * copies].double() - want_base).abs() <=
                     (n / 1000 + 32) * U32 * want_base)


@pytest.mark.parametrize("copies", [4, 8])
def test_two_sublayers_on_restored_streams(hc, copies):
    """A training step whose forward pass goes on from each stream as it was kept: what the mix
    numbers saw is what the backward pass reads, so that only roundings to bf16 along the way are
    left (y, out, dout, dy, each boundary's gradient: ten at most, each at most UBF and at random,
    half of that in the 2-norm; a parameter's gradient meets those of its sublayer's way up and of
    the way down)."""
    n, d, mix = 160, 256, (2 + copies) * copies
    g = t.gen(copies)
    A = [torch.randn(d, d, generator=g) * d ** -0.5 for _ in range(2)]
    P = [dict(w=torch.randn(mix, copies * d, generator=g) * (copies * d) ** -0.5,
              scale=0.5 + torch.rand(3, generator=g), base=torch.randn(mix, generator=g))
         for _ in range(2)]
    x0, top = t.bf16((n, copies, d), g), t.bf16((n, copies, d), g, 2.0 ** -6)

    ck = hc.hc_checkpoint(x0.cuda())
    keep = []
    for i in range(2):
        p = {k: v.cuda() for k, v in P[i].items()}
        x = hc.hc_restore(*ck)
        y, pre, post, comb, m = hc.hc_mixes_pre(x, p["w"], p["scale"], p["base"], want_mixes=True)
        out = (y.float() @ A[i].cuda()).to(torch.bfloat16)
        keep.append((ck, m, pre, post, comb, p))
        ck = hc.hc_post_checkpoint(out, x, post, comb)[1:]
    grad, got = top.cuda(), []
    for i in (1, 0):
        ck, m, pre, post, comb, p = keep[i]
        y = hc.hc_pre_restore(*ck, pre)
        out = (y.float() @ A[i].cuda()).to(torch.bfloat16)
        dout, dpost, dcomb, _ = hc.hc_post_backward(grad, out, ck, post, comb)
        dA = y.float().t() @ dout.float()
        dy = (dout.float() @ A[i].cuda().t()).to(torch.bfloat16)
        grad, dw, ds, db = hc.hc_mixes_pre_backward(dy, ck, m, p["w"], p["scale"], p["base"],
                                                    dpost, dcomb, dstream=grad, dx=grad)
        got.append((dA, dw, ds, db))

    xs = ref.values(keep[0][0]).requires_grad_()
    cur, leaves = xs, []
    for i in range(2):
        a = A[i].double().requires_grad_()
        w, s, b = (P[i][k].double().requires_grad_() for k in ("w", "scale", "base"))
        leaves += [a, w, s, b]
        y, _, po, co, _ = ref.mixes_pre(cur, w, s, b, 20, 1e-6, NORM_EPS)
        nxt = ref.post(y @ a, cur, po, co)
        cur = nxt if i == 1 else nxt + (ref.values(keep[1][0]) - nxt).detach()
    grads = torch.autograd.grad((cur * top.double()).sum(), [xs] + leaves)
    off = lambda a, b: float((a.cpu().double() - b).norm() / b.norm())  # noqa: E731
    tol = 10 * UBF / 2
    assert off(grad, grads[0]) <= tol
    for i, part in zip((1, 0), got):
        for a, b in zip(part, grads[1 + 4 * i:5 + 4 * i]):
            assert off(a, b) <= 2 * tol, i


@pytest.mark.parametrize("n,d,k8", [(200, 336, True), (129, 328, False), (1500, 1040, True)])
def test_in_place_on_the_streamed_path(hc, n, d, k8):
    # dx over dstream where tiles end past the last channel and the last token
    c = t.pre_case(hc, n, 4, d, k8)
    want = t.run_pre(hc, c)
    t.check_pre(want, c)
    buf = c["dstream"].clone()
    got = t.run_pre(hc, dict(c, dstream=buf), dx=buf)
    assert got[0] is buf
    for a, b in zip(got, want):
        assert torch.equal(a, b)
