"""Each input of hc_norm, hc_embed and their gradients written by the call directly before (GPU):
those launches overlap, so nothing of the input may be read before that call is done."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ROUNDS = 6


@pytest.fixture(scope="module")
def hc():
    import sinkhorn_mixing_gb300 as lib
    lib.lib()
    yield lib
    assert lib.hc_device_error(clear=True) == 0


def rand(seed, *shape, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def chained(make, use):
    """`make` writes an input, `use` reads it at once; the same with the device idle in between.
    The input's memory holds another call's numbers before."""
    for i in range(ROUNDS):
        torch.cuda.synchronize()
        got = use(make(i))
        made = make(i)
        torch.cuda.synchronize()
        for a, b in zip(got, use(made)):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("d", [128, 1000, 5120, 20480, 20488])
@pytest.mark.parametrize("center", [False, True])
def test_weights_and_biases(hc, d, center):
    """The last of many rows that hc_norm has just written."""
    rows = 40_000_000 // d
    many, out = rand(1, rows, d), torch.empty(rows, d, device="cuda")
    x, dy = rand(2, 300, d, dtype=BF16), rand(3, 300, d, dtype=BF16)
    factors = [rand(10 + i, d) for i in range(ROUNDS)]
    kw = dict(eps=1e-5, center=center)

    def make(i):
        return hc.hc_norm(many, factors[i], y=out)

    def use(y):
        return [hc.hc_norm(x, y[-1], y[-2], **kw)]

    def use_back(y):
        return hc.hc_norm_backward(dy, x, y[-1], want_dbias=True, **kw)

    chained(make, use)
    chained(make, use_back)


@pytest.mark.parametrize("d", [128, 5120, 20480, 20488])
def test_rows(hc, d):
    """x and dy that the call before has written, and a weight that the gradient's last launch has."""
    rows = 30_000_000 // d
    x, dy = rand(1, rows, d, dtype=BF16), rand(2, rows, d, dtype=BF16)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw = torch.empty(d, device="cuda")
    factors = [rand(10 + i, d) for i in range(ROUNDS)]
    kw = dict(eps=1e-5, center=True)
    ws = torch.empty(hc.hc_norm_backward_bytes(rows, d), dtype=torch.uint8, device="cuda")

    def make(i):
        return hc.hc_norm(x, factors[i], y=y, **kw)

    def use(z):
        return [hc.hc_norm(z, **kw)]

    def use_back(z):
        return hc.hc_norm_backward(dy, z, want_dbias=True, **kw)

    def use_dy(z):
        return hc.hc_norm_backward(z, x, want_dbias=True, **kw)

    for f in (use, use_back, use_dy):
        chained(make, f)

    def make_dw(i):
        return hc.hc_norm_backward(dy, x, factors[i], dx=dx, dweight=dw, workspace=ws, **kw)[1]

    def use_dw(w):
        return [hc.hc_norm(x[:40], w, **kw)]

    chained(make_dw, use_dw)


@pytest.mark.parametrize("n", [700, 6000])
def test_tables_and_ids(hc, n):
    """A table that its gradient's call has just written, ids that hc_norm has (a weight of zeros
    leaves the bias, whose bits are the ids), a stream's gradient that hc_embed has."""
    d, vocab = 1024, 20000
    g = torch.Generator().manual_seed(n)
    ids = torch.randint(0, vocab, (n,), generator=g, dtype=torch.int32).cuda()
    dx = rand(2, n, 4, d, dtype=BF16)
    table, dtable = rand(3, vocab, d), torch.empty(vocab, d, device="cuda")
    ws = torch.empty(hc.hc_embed_backward_bytes(n, d, vocab), dtype=torch.uint8, device="cuda")

    def make(i):
        return hc.hc_embed_backward(dx, ids, vocab, scale=1.0 + i, dtable=dtable, workspace=ws)

    def use(t):
        return [hc.hc_embed(ids, t)]

    chained(make, use)
    # as many ids as a row has channels, the last row's
    rows, width = 4000, 8 * (n // 8)
    many, out, zero = rand(4, rows, width), torch.empty(rows, width, device="cuda"), \
        torch.zeros(width, device="cuda")
    some = [torch.randint(-1, vocab, (width,), generator=g, dtype=torch.int32).cuda()
            for _ in range(ROUNDS)]

    def make_ids(i):
        return hc.hc_norm(many, zero, some[i].clamp(min=0).view(F32), y=out)[-1].view(torch.int32)

    def use_ids(v):
        return [hc.hc_embed(v, table),
                hc.hc_embed_backward(dx[:width], v, vocab)]

    def use_ids_back(v):
        return [hc.hc_embed_backward(dx[:width], v, vocab)]

    chained(make_ids, use_ids)
    chained(make_ids, use_ids_back)
    for i in range(ROUNDS):
        assert torch.equal(make_ids(i), some[i].clamp(min=0))

    x = torch.empty(n, 4, d, dtype=BF16, device="cuda")

    def make_dx(i):
        return hc.hc_embed(ids, table, scale=1.0 + i, x=x)

    def use_dx(v):
        return [hc.hc_embed_backward(v, ids, vocab),
                hc.hc_embed_backward(v, ids, vocab, dtable=table.clone(), accumulate=True)]

    chained(make_dx, use_dx)
