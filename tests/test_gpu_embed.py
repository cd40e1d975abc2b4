"""hc_embed and hc_embed_backward against their definitions (GPU)."""
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


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ids as they occur: all alike, all different, in runs, a few frequent ones, none in the table
def make_ids(kind, n, vocab, g):
    if kind == "same":
        return torch.full((n,), vocab - 1)
    if kind == "distinct":
        return torch.randperm(max(n, vocab), generator=g)[:n] % vocab
    if kind == "runs":
        return (torch.arange(n) // 7) % vocab
    if kind == "none":
        return torch.where(torch.arange(n) % 2 == 0, -1, vocab)
    ids = (vocab * torch.rand(n, generator=g) ** 4).long().clamp(max=vocab - 1)
    if kind == "padded":
        ids[torch.rand(n, generator=g) < 0.3] = -1
        ids[torch.rand(n, generator=g) < 0.1] = vocab
        ids[torch.rand(n, generator=g) < 0.1] = 2 ** 31 - 1
        ids[torch.rand(n, generator=g) < 0.05] = -2 ** 31
    return ids


KINDS = ["same", "distinct", "runs", "none", "frequent", "padded"]


def inside(ids, vocab):
    return (ids >= 0) & (ids < vocab)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("copies", [1, 4, 8])
@pytest.mark.parametrize("n,d,vocab", [(1, 8, 1), (3, 24, 5), (64, 5120, 300), (257, 1032, 1000),
                                       (5000, 72, 100)])
def test_embed(hc, n, d, vocab, copies, id_type, dtype):
    """scale * row is one product in binary32 and one rounding: equal in every bit."""
    g = gen(n + d)
    table = torch.randn(vocab, d, generator=g).to(dtype)
    for kind in ("padded", "frequent"):
        for scale in (1.0, d ** 0.5):
            ids = make_ids(kind, n, vocab, g)
            x = hc.hc_embed(ids.to(id_type).cuda(), table.cuda(), hc_mult=copies, scale=scale).cpu()
            row = table.float()[ids.clamp(0, vocab - 1)] * torch.tensor(scale, dtype=F32)
            row = torch.where(inside(ids, vocab)[:, None], row, torch.zeros(())).to(BF16)
            assert x.shape == (n, copies, d)
            assert torch.equal(x, row[:, None].expand(-1, copies, -1))


def test_embed_far_ids_and_special_numbers(hc):
    d = 64
    table = torch.randn(4, d, generator=gen(1))
    table[1, 3], table[2, 5], table[3, 7] = float("nan"), float("inf"), 3.4e38
    ids = torch.tensor([0, 1, 2, 3, 2 ** 32, 2 ** 32 + 1, -2 ** 63, 2 ** 63 - 1])
    x = hc.hc_embed(ids.cuda(), table.cuda(), hc_mult=4, scale=2.0).cpu()
    want = (table * 2.0).to(BF16)
    assert torch.equal(torch.isnan(x[1, :, 3]), torch.ones(4, dtype=torch.bool))
    assert torch.equal(x[2, 0], want[2]) and torch.equal(x[3, 0], want[3])
    assert not x[4:].any()


def test_embed_long_table_and_stream(hc):
    """More than 2^31 numbers in the table and in the stream."""
    d, vocab = 5120, (1 << 31) // 5120 + 50
    table = torch.zeros(vocab, d, dtype=BF16, device="cuda")
    row = torch.randn(d, generator=gen(2)).to(BF16)
    table[-1] = row.cuda()
    n = (1 << 31) // (8 * d) + 20
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    ids[-1] = vocab - 1
    x = hc.hc_embed(ids, table, hc_mult=8)
    assert torch.equal(x[-1].cpu(), row.expand(8, d)) and int(torch.count_nonzero(x[:-1])) == 0


def whole(shape, g):
    """Whole numbers whose sums stay whole in binary32, whatever their order."""
    return torch.randint(-4, 5, shape, generator=g).to(BF16)


# one tile of the sort and less, more tiles, more tiles than blocks would take one each; one digit
# and several; pieces of one token up to 32
SIZES = [(1, 8, 1), (2, 8, 2), (31, 64, 7), (33, 5120, 40), (64, 1032, 511), (65, 1032, 512),
         (700, 72, 600), (2047, 64, 3000), (2048, 40, 262143), (2049, 64, 262144), (4097, 520, 257),
         (5000, 5120, 64), (20011, 72, 1 << 20), (66000, 64, 50001)]


# either side of where the tokens are put in order another way
SIZES += [(7, 24, 3), (8, 24, 3), (9, 24, 3), (4095, 16, 4095), (4096, 16, 70000), (4097, 8, 3), (8191, 24, 300), (16400, 16, 1 << 19),
          (65535, 8, 131072), (65536, 16, 97), (65537, 8, 1000)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,d,vocab", SIZES)
def test_embed_backward_whole_numbers(hc, n, d, vocab, kind):
    """Every token's gradient arrives in its row, once: whole numbers, exact in any order."""
    g = gen(n + d + vocab)
    ids = make_ids(kind, n, vocab, g)
    copies = (1, 4, 8)[(n + d) % 3]
    dx = whole((n, copies, d), g)
    dx[~inside(ids, vocab)] = float("nan")          # not read
    id_type = torch.int64 if n % 2 else torch.int32
    idd, dxd = ids.to(id_type).cuda(), dx.cuda()
    ok = inside(ids, vocab)
    rows = ids[ok].unique()
    got = hc.hc_embed_backward(dxd, idd, vocab, dtable=torch.full((vocab, d), 9.0, device="cuda"))
    want = torch.zeros(vocab, d).index_add_(0, ids[ok], dx[ok].float().sum(1))
    assert torch.equal(got.cpu(), want)
    # added to what is there; other rows are left alone
    base = torch.full((vocab, d), float("nan"), device="cuda")
    base[rows.cuda()] = 3.0
    hc.hc_embed_backward(dxd, idd, vocab, dtable=base, accumulate=True)
    base = base.cpu()
    assert torch.equal(base[rows], want[rows] + 3.0)
    left = torch.ones(vocab, dtype=torch.bool)
    left[rows] = False
    assert torch.isnan(base[left]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("copies", [1, 4, 8])
@pytest.mark.parametrize("n,d,vocab", [(5, 40, 9), (333, 1000, 50), (3001, 264, 700)])
def test_embed_backward(hc, n, d, vocab, copies, dtype):
    g = gen(n + d + copies)
    ids = make_ids("padded", n, vocab, g)
    dx = (torch.randn(n, copies, d, generator=g) * 2.0 ** -5).to(BF16)
    scale = 1.75
    want, mag = ref.embed_backward(ids, dx.double(), vocab, scale)
    got = hc.hc_embed_backward(dx.cuda(), ids.cuda(), vocab, scale=scale, dtype=dtype)
    off = ref.embed_chain(n) * ref.U32 * mag
    half, tiny = ref.HALF[dtype] * (1 + 1e-3), ref.TINY[dtype]
    assert got.dtype == dtype
    assert torch.all((got.cpu().double() - want).abs() <= off + half * want.abs() + tiny)
    base = torch.randn(vocab, d, generator=g).to(dtype)
    got = hc.hc_embed_backward(dx.cuda(), ids.cuda(), vocab, scale=scale, dtable=base.cuda(),
                               accumulate=True).cpu().double()
    want2 = want + base.double()
    tol = off + ref.U32 * 1.01 * want2.abs() + half * want2.abs() + tiny
    assert torch.all((got - want2).abs() <= tol)
    # against differences of the forward definition along a direction: it is linear
    u = torch.randn(vocab, d, generator=g, dtype=torch.float64)
    ok = inside(ids, vocab)
    along = (u[ids[ok]][:, None] * scale * dx[ok].double()).sum()
    tol = ((got - want2).abs() + off + half * want.abs()).mul(u.abs()).sum() + 1e-9
    assert abs(float(((got - base.double()) * u).sum() - along)) <= float(tol)


@pytest.mark.parametrize("n,d,vocab", [(40, 72, 9), (3001, 264, 700), (9000, 1032, 50)])
def test_same_bits_streams_and_graph(hc, n, d, vocab):
    g = gen(n)
    ids = make_ids("frequent", n, vocab, g).cuda()
    dx = torch.randn(n, 4, d, generator=g).to(BF16).cuda()
    want = hc.hc_embed_backward(dx, ids, vocab)
    for _ in range(3):
        assert torch.equal(hc.hc_embed_backward(dx, ids, vocab), want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = hc.hc_embed_backward(dx, ids, vocab, stream=side)
    table = torch.randn(vocab, d, generator=g).cuda()
    torch.cuda.synchronize()
    x = hc.hc_embed(ids, table, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(x, hc.hc_embed(ids, table))
    # captured, replayed on new ids and gradients
    ws = torch.empty(hc.hc_embed_backward_bytes(n, d, vocab), dtype=torch.uint8, device="cuda")
    out, xs = torch.empty(vocab, d, device="cuda"), torch.empty_like(dx)
    idb, dxb = ids.clone(), dx.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hc.hc_embed(idb, table, x=xs)
        hc.hc_embed_backward(dxb, idb, vocab, dtable=out, workspace=ws)
        hc.hc_embed_backward(dxb, idb, vocab, dtable=out, workspace=ws, accumulate=True)
    ids2 = make_ids("padded", n, vocab, g).cuda()
    dx2 = whole((n, 4, d), g).cuda()
    for i, x in ((ids, dx), (ids2, dx2)):
        idb.copy_(i), dxb.copy_(x)
        graph.replay()
        once = hc.hc_embed_backward(x, i, vocab)
        assert torch.equal(xs, hc.hc_embed(i, table))
        assert torch.equal(out, hc.hc_embed_backward(x, i, vocab, dtable=once, accumulate=True))


def test_guards_and_empty(hc):
    n, d, vocab = 77, 136, 31
    g = gen(8)
    ids = make_ids("padded", n, vocab, g).cuda()
    dx = whole((n, 4, d), g).cuda()
    for dtype in TYPES:
        big = torch.full((vocab * d + 128,), 7.0, dtype=dtype, device="cuda")
        need = hc.hc_embed_backward_bytes(n, d, vocab)
        ws = torch.full((need + 512,), 5, dtype=torch.uint8, device="cuda")
        out = big[64:64 + vocab * d].view(vocab, d)
        hc.hc_embed_backward(dx, ids, vocab, dtable=out, workspace=ws[256:256 + need])
        assert bool((big[:64] == 7).all()) and bool((big[64 + vocab * d:] == 7).all())
        assert bool((ws[:256] == 5).all()) and bool((ws[256 + need:] == 5).all())
        x = torch.full((n * 4 * d + 128,), 7.0, dtype=BF16, device="cuda")
        hc.hc_embed(ids, out, x=x[64:64 + n * 4 * d].view(n, 4, d))
        assert bool((x[:64] == 7).all()) and bool((x[64 + n * 4 * d:] == 7).all())
        none = torch.empty(0, dtype=torch.int64, device="cuda")
        assert hc.hc_embed(none, out).shape == (0, 4, d)
        left = out.clone()
        hc.hc_embed_backward(dx[:0], none, vocab, dtable=out, accumulate=True)
        assert torch.equal(out, left)
        hc.hc_embed_backward(dx[:0], none, vocab, dtable=out)
        assert not out.any()
    # shapes as a batch has them
    x = hc.hc_embed(ids[:76].view(4, 19), torch.ones(vocab, d, device="cuda"), hc_mult=8)
    assert x.shape == (4, 19, 8, d)
    a = hc.hc_embed_backward(dx[:76].view(4, 19, 4, d), ids[:76].view(4, 19), vocab)
    assert torch.equal(a, hc.hc_embed_backward(dx[:76], ids[:76].contiguous(), vocab))
    # ids that start at an odd place
    assert torch.equal(hc.hc_embed_backward(dx[1:], ids[1:], vocab),
                       hc.hc_embed_backward(dx[1:], ids[1:].clone(), vocab))


def test_embed_backward_long(hc):
    """More than 2^31 gradients and table entries."""
    d, n = 5120, (1 << 31) // (8 * 5120) + 20
    vocab = (1 << 31) // d + 50
    dx = torch.zeros(n, 8, d, dtype=BF16, device="cuda")
    ids = torch.arange(n, device="cuda") % 1000
    ids[-1] = vocab - 1
    dx[-1], dx[-2] = 1.0, 2.0
    got = hc.hc_embed_backward(dx, ids, vocab, dtype=BF16)
    assert torch.all(got[-1] == 8.0) and torch.all(got[(n - 2) % 1000] == 16.0)
    assert int(torch.count_nonzero(got)) == 2 * d


@pytest.mark.parametrize("n", [3000, 9000])
def test_embed_backward_most_rows(hc, n):
    """Ids of all 31 bits; only the rows that tokens name are touched."""
    vocab, d = (1 << 31) - 2, 8
    g = gen(n)
    ids = torch.randint(0, vocab, (n,), generator=g)
    ids[::3], ids[5], ids[6] = ids[0].item(), vocab - 1, 0
    dx = whole((n, 1, d), g)
    table = torch.empty(vocab, d, dtype=BF16, device="cuda")
    rows, at = ids.unique(return_inverse=True)
    table[rows.cuda()] = 1.0
    hc.hc_embed_backward(dx.cuda(), ids.cuda(), vocab, dtable=table, accumulate=True)
    want = torch.ones(rows.numel(), d).index_add_(0, at, dx[:, 0].float()).to(BF16)
    assert torch.equal(table[rows.cuda()].cpu(), want)
    x = hc.hc_embed(ids.to(torch.int32).cuda(), table, hc_mult=1)
    assert torch.equal(x[:, 0].cpu(), want[at])


def test_refusals(hc):
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    table = torch.zeros(9, 64, device="cuda")
    dx = torch.zeros(4, 4, 64, dtype=BF16, device="cuda")
    with pytest.raises(hc.HcError, match="UNSUPPORTED"):
        hc.hc_embed(ids, table, hc_mult=2)
    with pytest.raises(hc.HcError, match="INVALID"):
        hc.hc_embed(ids, table, scale=float("nan"))
    with pytest.raises(TypeError):
        hc.hc_embed(ids, table.double())
    with pytest.raises(ValueError):
        hc.hc_embed(ids.cpu(), table)
    with pytest.raises(ValueError):
        hc.hc_embed(ids, table.t().contiguous().t())
    with pytest.raises(ValueError):
        hc.hc_embed_backward(dx[:3], ids, 9)
    with pytest.raises(ValueError):
        hc.hc_embed_backward(dx, ids, 9, accumulate=True)
    with pytest.raises(ValueError):
        hc.hc_embed_backward(dx, ids, 9, dtable=table[:8])
    with pytest.raises(hc.HcError, match="INVALID"):
        hc.hc_embed_backward(dx, ids, 0)
    with pytest.raises(hc.HcError, match="INVALID"):
        hc.hc_embed_backward(dx, ids, 9, workspace=torch.empty(0, dtype=torch.uint8,
                                                               device="cuda"))
