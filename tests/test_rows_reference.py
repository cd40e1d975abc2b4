"""The 64-bit forms of the norm and the embedding against automatic differentiation, differences
and torch's own layer norm (CPU)."""
import pytest
import torch

import rows_reference as ref


def case(n, d, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(n, d) * torch.exp(r(n, 1)) + r(n, 1), r(n, d), 1 + r(d), r(d)


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_norm_gradients(center, weighted):
    x, dy, w, b = case(5, 24, 3)
    w, b = (w, b) if weighted else (None, None)
    leaves = [t.clone().requires_grad_() for t in (x, w, b) if t is not None]
    y = ref.norm(leaves[0], *(leaves[1:] if weighted else (None, None)), center, 1e-5)
    if center:
        want = torch.nn.functional.layer_norm(x, (24,), w, b, 1e-5)
        assert torch.allclose(y.detach(), want, rtol=1e-12, atol=1e-12)
    got = ref.norm_backward(dy, x, w, center, 1e-5)
    for a, g in zip(got, torch.autograd.grad(y, leaves, dy)):
        assert torch.allclose(a, g, rtol=1e-11, atol=1e-12)
    # against differences along a direction of each input
    dirs = [torch.randn(t.shape, dtype=torch.float64) for t in (x,) + ((w, b) if weighted else ())]
    for i, u in enumerate(dirs):
        args = [x] + ([w, b] if weighted else [None, None])
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + 1e-6 * u, args[i] - 1e-6 * u
        diff = ((ref.norm(*hi, center, 1e-5) - ref.norm(*lo, center, 1e-5)) * dy).sum() / 2e-6
        assert abs(float(diff - (got[i] * u).sum())) <= 1e-6 * (1 + abs(float(diff)))


def test_embed_gradient():
    g = torch.Generator().manual_seed(1)
    ids = torch.tensor([3, -1, 0, 3, 7, 9, 3])
    dx = torch.randn(7, 4, 8, generator=g, dtype=torch.float64)
    table = torch.randn(7, 8, generator=g, dtype=torch.float64).requires_grad_()
    ok = (ids >= 0) & (ids < 7)
    x = (1.5 * table[ids[ok]])[:, None].expand(-1, 4, -1)
    want, = torch.autograd.grad(x, table, dx[ok])
    got, mag = ref.embed_backward(ids, dx, 7, 1.5)
    assert torch.allclose(got, want, rtol=1e-13)
    assert torch.all(mag >= got.abs())
