"""The 64-bit forms that the training operators are tested against, themselves held to differences
and to torch's own 8-bit type (CPU)."""
import numpy as np
import pytest
import torch

import train_reference as ref


def test_e4m3_table_is_torch_s():
    c = torch.arange(256, dtype=torch.uint8)
    t = c.view(torch.float8_e4m3fn).double().numpy()
    v = ref.e4m3_values()
    assert np.array_equal(np.isnan(t), np.isnan(v))
    ok = ~np.isnan(v)
    assert np.array_equal(t[ok], v[ok])


def test_checkpoint_form():
    bits = np.arange(65536, dtype=np.uint16).reshape(-1, 64)     # every bf16 number
    codes, scales = ref.checkpoint(bits)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    v = ref.values((torch.from_numpy(codes), torch.from_numpy(scales)))
    f = x.double()
    fin = torch.isfinite(f)
    assert torch.equal(torch.isnan(v), ~fin)
    # every row spans half an exponent's range: relative error at most half a step
    err = (v - f)[fin].abs()
    assert torch.all(err <= 2.0 ** -4 * f[fin].abs() + 2.0 ** -136)
    # nothing saturates: the largest code of a block is what its largest number rounds to
    assert scales.min() == 1 and scales.max() <= 247
    # torch rounds to e4m3 as the table's nearest-even does
    s = np.repeat(np.exp2(127.0 - scales.astype(np.float64)), 32, 1)
    s = torch.from_numpy(s)
    over = torch.where(s == 2.0 ** -120, (f * s).clamp(-240, 240), f * s)
    t = over.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(t[fin.numpy()], codes[fin.numpy()])
    assert torch.equal(v[fin], v[fin].to(torch.bfloat16).double())


@pytest.mark.parametrize("hc", [4, 8])
def test_gradients_against_differences(hc):
    g = torch.Generator().manual_seed(3)
    n, d, iters, eps, norm_eps = 3, 16, 20, 1e-6, 1e-6
    mix = (2 + hc) * hc
    rn = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w = rn(n, hc, d), rn(mix, hc * d) * (hc * d) ** -0.5
    scale, base = rn(3) + 1, rn(mix)
    dy, dpost, dcomb, ds = rn(n, d), rn(n, hc), rn(n, hc, hc), rn(n, hc, d)
    m = ref.mixes(x, w, norm_eps)
    comb0 = ref.split(ref.logits(m, scale, base, hc), hc, iters, eps)[2]
    (dx, dw, dscale, dbase), _ = ref.mixes_pre_backward(dy, x, m, w, scale, base, dpost, dcomb, ds,
                                                        iters, eps, norm_eps)

    def loss(x, w, scale, base):
        y, _, po, co, _ = ref.mixes_pre(x, w, scale, base, iters, eps, norm_eps)
        past = torch.einsum("njk,njc->nkc", comb0, x)
        return (y * dy).sum() + (po * dpost).sum() + (co * dcomb).sum() + (past * ds).sum()

    at = [x, w, scale, base]
    for i, grad in enumerate((dx, dw, dscale, dbase)):
        v = rn(*at[i].shape)
        h = 1e-5
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * v, at[i] - h * v
        num = (loss(*up) - loss(*down)) / (2 * h)
        assert abs(num - (grad * v).sum()) <= 1e-7 * (grad * v).abs().sum()
