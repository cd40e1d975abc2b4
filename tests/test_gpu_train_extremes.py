"""hc_mixes_pre_backward at the ends of binary32's range (GPU)."""
import pytest
import torch

import test_gpu_train as t
import train_reference as ref

pytestmark = pytest.mark.gpu
U32, UBF = ref.U32, ref.UBF


@pytest.fixture(scope="module")
def hc():
    import sinkhorn_mixing_gb300 as lib
    lib.lib()
    yield lib
    assert lib.hc_device_error(clear=True) == 0


@pytest.mark.parametrize("copies,n,d", [(4, 40, 96), (4, 200, 96), (8, 40, 96)])
def test_zeros_in_a_block_of_large_numbers(hc, copies, n, d):
    # A block whose scale's square is above binary32's range, with channels of zero in it.  The
    # squares' sum is infinite and r = 0, whether the stream is kept in 8 bits or as the bf16
    # numbers that these stand for.
    c = t.pre_case(hc, n, copies, d, False)
    c["x"][3, 1, :32] = 0
    c["x"][3, 1, 2] = 2.0 ** 100
    c["mixes"][3] = 0
    kept = hc.hc_checkpoint(c["x"])
    got = t.run_pre(hc, dict(c, x=kept))
    want = t.run_pre(hc, dict(c, x=hc.hc_restore(*kept)))
    for a, b in zip(got, want):
        assert bool(torch.isfinite(b).all()) and bool(torch.isfinite(a).all())
    # Scales are powers of two, so both sum the same numbers; sums of their parts may be taken in
    # another order: dx's rounding to bf16 twice, and binary32's over n tokens in dW
    x = ref.values(kept)
    a, b = got[0].cpu().double(), want[0].cpu().double()
    assert torch.all((a - b).abs() <= 2 * UBF * b.abs() + 2.0 ** -10 * b.abs().amax(2, keepdim=True))
    for a, b in zip(got[1:], want[1:]):
        assert float((a - b).abs().max()) <= 2 * (n + 32) * U32 * n * float(b.abs().max())
    # the token itself: its terms without r (r = 0), which are pre dy + comb dstream
    pre, _, comb = ref.split(c["base"].cpu().double()[None], copies, 20, 1e-6)
    dy, ds = c["dy"][3].cpu().double(), c["dstream"][3].cpu().double()
    dx = pre[0][:, None] * dy + comb[0] @ ds
    mag = pre[0][:, None] * dy.abs() + comb[0] @ ds.abs()
    tol = UBF * dx.abs() + (ref.split_tolerance(20) + (16 + copies) * U32) * mag
    assert torch.all((got[0][3].cpu().double() - dx).abs() <= tol)
    assert bool((x[3, 1, 2] == 2.0 ** 100).all())


@pytest.mark.parametrize("copies,n", [(4, 40), (4, 200), (8, 40)])
@pytest.mark.parametrize("k8", [True, False])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_gradient_of_one_mix_number(hc, copies, n, k8, sign):
    # du of one mix number is infinite: its row of dW is du x summed, infinite with x's sign (NaN
    # where x is 0), and the other rows are as they were
    c = t.pre_case(hc, n, copies, 96, k8)
    plain = t.run_pre(hc, c)
    c["dpost"][5, 2] = sign * float("inf")
    got = t.run_pre(hc, c)
    row = copies + 2
    x = ref.values(c["x"])[5].flatten()
    dw = got[1].cpu().double()
    keep = [i for i in range(dw.shape[0]) if i != row]
    assert torch.equal(got[1][keep], plain[1][keep])
    assert torch.equal(dw[row][x != 0], sign * x[x != 0].sign() * float("inf"))
    assert bool(torch.isnan(dw[row][x == 0]).all())
    assert float(got[3][row]) == sign * float("inf")
    tokens = [i for i in range(n) if i != 5]
    assert torch.equal(got[0][tokens], plain[0][tokens])
