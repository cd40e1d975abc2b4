"""hc_embed_backward against the 64-bit sums and against differences, with bounds that hold nothing
but the roundings it needs (GPU; test_rows_bounds.py shows what they let pass)."""
import pytest
import torch

import rows_reference as ref
import test_gpu_embed as embed

pytestmark = pytest.mark.gpu
hc = embed.hc


@pytest.mark.parametrize("dtype", embed.TYPES)
@pytest.mark.parametrize("n,d,vocab,copies", [(1, 8, 3, 4), (9, 40, 9, 8), (333, 1000, 50, 4),
                                              (1537, 264, 700, 8), (4096, 72, 97, 1),
                                              (9001, 136, 300, 4)])
def test_embed_backward(hc, n, d, vocab, copies, dtype):
    g = embed.gen(n + d)
    for kind in ("frequent", "padded", "same"):
        ids = embed.make_ids(kind, n, vocab, g)
        dx = (torch.randn(n, copies, d, generator=g) * 2.0 ** -5).to(torch.bfloat16)
        base = torch.randn(vocab, d, generator=g).to(dtype)
        got = hc.hc_embed_backward(dx.cuda(), ids.cuda(), vocab, scale=1.75, dtype=dtype)
        ref.check_embed_backward(got, None, ids, dx, vocab, 1.75, dtype)
        got = hc.hc_embed_backward(dx.cuda(), ids.cuda(), vocab, scale=-0.3, dtable=base.cuda(),
                                   accumulate=True)
        scale = float(torch.tensor(-0.3))       # as the call takes it, in binary32
        ref.check_embed_backward(got, base, ids, dx, vocab, scale, dtype)
