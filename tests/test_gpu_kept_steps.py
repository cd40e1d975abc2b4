"""The training step of test_gpu_token_steps.py against the same step in 64 bits, every part of
which reads what the calls read: the forward pass the stream, the backward pass what was kept of it
(GPU).  So kept streams in 8 bits cost no tolerance, and what is left is rounding to bf16."""
import pytest
import torch

import rows_reference as rows
import test_gpu_token_steps as steps
import train_reference as ref

pytestmark = pytest.mark.gpu
hc = steps.hc
SPLIT = (20, 1e-6, steps.NORM_EPS)
# A number passes through at most 14 roundings to bf16 on its way down (y, its norm, out and, of the
# gradient, dout, dh, dy and dx in each of two layers; y, dy and the stream's gradient at the end),
# each by UBF at most and by half of that in the 2-norm; 20 allow for the factors that differ from
# one, such as the norms'.  A layer's parameters have products of two such numbers.
TOL = 20 * ref.UBF / 2


def layer(q, x, kept):
    """A layer's forward pass and, from `kept`, its recomputed sublayer, in 64 bits."""
    w, s, b, nw, A = (q[k].double() for k in ("w", "scale", "base", "norm", "A"))
    y, pre, post, comb, m = ref.mixes_pre(x, w, s, b, *SPLIT)
    x = ref.post(rows.norm(y, nw, None, False, 1e-20) @ A, x, post, comb)
    y = torch.einsum("nj,njc->nc", pre, kept)
    h = rows.norm(y, nw, None, False, 1e-20)
    return x, (y, h, h @ A, post, comb, m)


def layer_backward(q, kept, again, grad):
    w, s, b, nw, A = (q[k].double() for k in ("w", "scale", "base", "norm", "A"))
    y, h, out, post, comb, m = again
    (dout, dpost, dcomb, _), _ = ref.post_backward(grad, out, kept, post, comb)
    dy, dnorm, _ = rows.norm_backward(dout @ A.t(), y, nw, False, 1e-20)
    (dx, dw, ds, db), _ = ref.mixes_pre_backward(dy, kept, m, w, s, b, dpost, dcomb, grad, *SPLIT)
    return dx, (dnorm, h.t() @ dout, dw, ds, db)


@pytest.mark.parametrize("copies,n", [(4, 96), (8, 80), (4, 200)])
@pytest.mark.parametrize("k8", [False, True])
def test_step(hc, copies, n, k8):
    d, vocab, layers = 256, 40, 2
    ids, p, top = steps.model(copies, n, d, vocab, layers, copies + n)
    pc = steps.cuda(p)
    z, dfinal, dtable, got, kept = steps.step(hc, ids.cuda(), pc, top.cuda(), copies, k8)
    # the streams at the boundaries: the calls give the same bits each time
    xs = [hc.hc_embed(ids.cuda(), pc["table"], hc_mult=copies, scale=1.5)]
    for i in range(1, layers):
        xs.append(steps.step(hc, ids.cuda(), dict(pc, layers=pc["layers"][:i]), top.cuda(), copies,
                             k8)[4][-1])
    xs.append(kept[-1])
    kept[-1] = hc.hc_checkpoint(xs[-1]) if k8 else xs[-1]       # hc_post_checkpoint's bits
    torch.cuda.synchronize()
    xs, kept = [ref.values(x) for x in xs], [ref.values(k) for k in kept]

    def off(a, b):
        return float((a.detach().cpu().double() - b).norm() / b.norm())

    again = []
    for i, q in enumerate(p["layers"]):
        x, back = layer(q, xs[i], kept[i])
        assert off(xs[i + 1], x) <= TOL
        again.append(back)
    y = torch.einsum("nj,njc->nc", p["out"].double(), kept[-1])
    final = p["final"].double()
    assert off(z, rows.norm(y, final, None, False, 1e-20)) <= TOL
    dy, want_final, _ = rows.norm_backward(top.double(), y, final, False, 1e-20)
    assert off(dfinal, want_final) <= TOL
    grad = p["out"].double()[..., None] * dy[:, None]
    for i in reversed(range(layers)):
        grad, wants = layer_backward(p["layers"][i], kept[i], again[i], grad)
        for a, b in zip(got[i], wants):
            assert off(a, b) <= 2 * TOL
    assert off(dtable, rows.embed_backward(ids, grad, vocab, 1.5)[0]) <= TOL
