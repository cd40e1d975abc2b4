"""What a table's gradient is held to in the tests: the rounded 64-bit sums pass, a planted mistake
does not (CPU)."""
import pytest
import torch

import rows_reference as ref

VOCAB, SCALE = 50, 1.75


def case(n=333, d=40, copies=4):
    g = torch.Generator().manual_seed(n)
    ids = (VOCAB * torch.rand(n, generator=g) ** 4).long()
    ids[::7] = -1
    return ids, (torch.randn(n, copies, d, generator=g) * 2.0 ** -5).to(torch.bfloat16)


def halved(got, ids, dx):
    return got / 2


def nothing(got, ids, dx):
    return torch.zeros_like(got)


def a_token_left_out(got, ids, dx):
    got = got.clone()
    got[ids[1]] -= SCALE * dx[1].double().sum(0)
    return got


def a_token_twice(got, ids, dx):
    got = got.clone()
    got[ids[2]] += SCALE * dx[2].double().sum(0)
    return got


def a_copy_left_out(got, ids, dx):
    return got - ref.embed_backward(ids, dx[:, :1].double(), VOCAB, SCALE)[0]


def rows_one_further(got, ids, dx):
    return got.roll(1, 0)


def without_the_scale(got, ids, dx):
    return got / SCALE


def added_up_in_sixteen_bits(got, ids, dx):
    out = torch.zeros_like(got)
    for i, v in zip(ids.tolist(), dx.double().sum(1)):
        if i >= 0:
            out[i] = (out[i] + SCALE * v).to(torch.bfloat16).double()
    return out


MISTAKES = [halved, nothing, a_token_left_out, a_token_twice, a_copy_left_out, rows_one_further,
            without_the_scale, added_up_in_sixteen_bits]


@pytest.mark.parametrize("added", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_embed_backward_bound(dtype, added):
    ids, dx = case()
    want, _ = ref.embed_backward(ids, dx.double(), VOCAB, SCALE)
    base = None
    if added:
        base = torch.randn(want.shape, generator=torch.Generator().manual_seed(1)).to(dtype)

    def check(grad):
        total = grad if base is None else grad + base.double()
        ref.check_embed_backward(total.to(dtype), base, ids, dx, VOCAB, SCALE, dtype)

    check(want)
    for mistake in MISTAKES:
        # the sums' roundings to 16 bits hide behind the one rounding of large numbers to them
        if mistake is added_up_in_sixteen_bits and added and dtype != torch.float32:
            continue
        with pytest.raises(AssertionError):
            check(mistake(want, ids, dx))
