"""A training step from token ids to the normed output and back, as a user would run it (GPU)."""
import pytest
import torch

import rows_reference as rows
import test_gpu_train as t
import train_reference as ref

pytestmark = pytest.mark.gpu
UBF, NORM_EPS = ref.UBF, t.NORM_EPS
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def hc():
    import sinkhorn_mixing_gb300 as lib
    lib.lib()
    yield lib
    assert lib.hc_device_error(clear=True) == 0


def model(copies, n, d, vocab, layers, seed):
    g = t.gen(seed)
    mix = (2 + copies) * copies
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    ids = (vocab * torch.rand(n, generator=g) ** 3).long()
    ids[::17] = -1
    p = dict(table=r(vocab, d).to(BF16), final=1 + 0.25 * r(d),
             out=torch.softmax(r(n, copies), 1),
             layers=[dict(w=r(mix, copies * d) * (copies * d) ** -0.5,
                          scale=0.5 + torch.rand(3, generator=g), base=r(mix),
                          norm=1 + 0.25 * r(d), A=r(d, d) * d ** -0.5) for _ in range(layers)])
    return ids, p, (r(n, d) * 2.0 ** -6).to(BF16)


def cuda(p):
    return {k: [cuda(q) for q in v] if isinstance(v, list) else v.cuda() for k, v in p.items()}


def step(hc, ids, p, top, copies, k8, scale=1.5):
    """Gradients of <normed output, top>: of the table, the norms, the matrices and the mixing.
    Streams are kept at each boundary, and each sublayer is recomputed from them."""
    x, keep = hc.hc_embed(ids, p["table"], hc_mult=copies, scale=scale), []
    ck = hc.hc_checkpoint(x) if k8 else x
    for q in p["layers"]:
        y, pre, post, comb, m = hc.hc_mixes_pre(x, q["w"], q["scale"], q["base"], want_mixes=True)
        h = hc.hc_norm(y, q["norm"])
        out = (h.float() @ q["A"]).to(BF16)
        keep.append((ck, m, pre, post, comb))
        if k8:
            x, c8, s8 = hc.hc_post_checkpoint(out, x, post, comb)
            ck = (c8, s8)
        else:
            x = hc.hc_post(out, x, post, comb)
            ck = x
    y = hc.hc_pre_restore(*ck, p["out"]) if k8 else hc.hc_pre(ck, p["out"])
    z = hc.hc_norm(y, p["final"])
    dy, dfinal, _ = hc.hc_norm_backward(top, y, p["final"])
    grad = (p["out"][..., None] * dy[:, None].float()).to(BF16)
    got = []
    for q, (ck, m, pre, post, comb) in zip(p["layers"][::-1], keep[::-1]):
        y = hc.hc_pre_restore(*ck, pre) if k8 else hc.hc_pre(ck, pre)
        h = hc.hc_norm(y, q["norm"])
        out = (h.float() @ q["A"]).to(BF16)
        dout, dpost, dcomb, _ = hc.hc_post_backward(grad, out, ck, post, comb)
        dA = h.float().t() @ dout.float()
        dh = (dout.float() @ q["A"].t()).to(BF16)
        dy, dnorm, _ = hc.hc_norm_backward(dh, y, q["norm"])
        grad, dw, ds, db = hc.hc_mixes_pre_backward(dy, ck, m, q["w"], q["scale"], q["base"], dpost,
                                                    dcomb, dstream=grad, dx=grad)
        got.append((dnorm, dA, dw, ds, db))
    dtable = hc.hc_embed_backward(grad, ids, p["table"].shape[0], scale=scale)
    return z, dfinal, dtable, got[::-1], [k[0] for k in keep] + [ck if not keep else x]


@pytest.mark.parametrize("copies,n", [(4, 96), (8, 80), (4, 200)])
@pytest.mark.parametrize("k8", [False, True])
def test_tokens_to_output_and_back(hc, copies, n, k8):
    d, vocab, layers = 256, 40, 2
    ids, p, top = model(copies, n, d, vocab, layers, copies + n)
    z, dfinal, dtable, got, kept = step(hc, ids.cuda(), cuda(p), top.cuda(), copies, k8)
    torch.cuda.synchronize()

    # the same step in 64 bits; each boundary's stream takes the value that was kept
    leaf = lambda a: a.double().requires_grad_()  # noqa: E731
    table, final = leaf(p["table"]), leaf(p["final"])
    ok = (ids >= 0)[:, None, None]
    cur = (1.5 * table[ids.clamp(min=0)])[:, None].expand(-1, copies, -1) * ok
    cur = cur + (ref.values(kept[0]) - cur).detach()
    leaves = []
    for i, q in enumerate(p["layers"]):
        w, s, b, nw, A = (leaf(q[k]) for k in ("w", "scale", "base", "norm", "A"))
        leaves += [nw, A, w, s, b]
        y, _, po, co, _ = ref.mixes_pre(cur, w, s, b, 20, 1e-6, NORM_EPS)
        nxt = ref.post(rows.norm(y, nw, None, False, 1e-20) @ A, cur, po, co)
        if i + 1 < layers:
            nxt = nxt + (ref.values(kept[i + 1]) - nxt).detach()
        cur = nxt
    y = torch.einsum("nj,njc->nc", p["out"].double(), cur)
    want_z = rows.norm(y, final, None, False, 1e-20)
    grads = torch.autograd.grad((want_z * top.double()).sum(), [table, final] + leaves)
    off = lambda a, b: float((a.cpu().double() - b).norm() / b.norm())  # noqa: E731
    # roundings to bf16 on the way up and down: y, h, out, the stream; dh, dy, dout, the stream's
    # gradient, for each of two sublayers and the end, each at most UBF and at random, half of that
    # in the 2-norm; 8-bit streams are the numbers above rounded to 2^-4 more, at random over
    # copies * d channels, in the mix numbers' and the last stream's values
    tol = 20 * UBF / 2 + (2.0 ** -4 * 4 if k8 else 0)
    assert off(z, want_z.detach()) <= tol
    assert off(dtable, grads[0]) <= tol and off(dfinal, grads[1]) <= tol
    assert not dtable.cpu()[~torch.isin(torch.arange(vocab), ids)].any()
    for a, b in zip([v for part in got for v in part], grads[2:]):
        assert off(a, b) <= 2 * tol


@pytest.mark.parametrize("n", [64, 300])
def test_captured_step(hc, n):
    """The whole step in a graph, replayed on new tokens: the bits of the eager calls."""
    ids, p, top = model(4, n, 256, 40, 2, n)
    other = model(4, n, 256, 40, 2, n + 1)[0].cuda()
    ids, p, top = ids.cuda(), cuda(p), top.cuda()
    flat = lambda s: [s[0], s[1], s[2]] + [v for part in s[3] for v in part]  # noqa: E731
    want = [flat(step(hc, i, p, top, 4, False)) for i in (ids, other)]
    buf = ids.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = flat(step(hc, buf, p, top, 4, False))
    for i, w in zip((ids, other), want):
        buf.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n,copies,d", [(5, 4, 64), (64, 4, 5120), (300, 8, 1024), (500, 4, 2048)])
def test_norm_is_the_fused_calls(hc, n, copies, d):
    """hc_norm of hc_mixes_pre's y against hc_mixes_pre_norm: the fused kernel takes the mean square
    before y's rounding to bf16, so a row's factor may differ by 2^-8 of the rounding at random over
    the row, and an element by a bf16 step where it lies next to a border."""
    g = t.gen(n + d)
    x = (t.bf16((n, copies, d), g).float() * torch.exp(torch.randn(n, 1, 1, generator=g))).to(BF16)
    mix = (2 + copies) * copies
    w = (torch.randn(mix, copies * d, generator=g) * (copies * d) ** -0.5).cuda()
    scale, base = torch.ones(3).cuda(), torch.randn(mix, generator=g).cuda()
    rms = (0.5 + torch.rand(d, generator=g)).cuda()
    y = hc.hc_mixes_pre(x.cuda(), w, scale, base)[0]
    a = hc.hc_norm(y, rms).float()
    b = hc.hc_mixes_pre_norm(x.cuda(), w, scale, base, rms)[0].float()
    step_ = 2.0 ** -7 * b.abs()             # a bf16 step, at least half of it and at most all
    assert torch.all((a - b).abs() <= 2 * step_)
    assert float(((a - b).abs() > 0).float().mean()) < 0.05
