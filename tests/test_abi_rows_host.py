"""Refusals of hc_norm, hc_embed and their gradients on the host: bad arguments return the
documented status before any CUDA call (the device pointers are fake addresses that nothing dereferences)."""
import ctypes
import math
import os
import shutil

import pytest

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA = 0, 1, 2, 3, 4
BF16, F16, F32 = 0, 1, 2
A, GAP = 1 << 20, 1 << 40

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


def no_gpu():
    import torch
    return not torch.cuda.is_available()


@pytest.fixture(scope="module")
def L():
    from sinkhorn_mixing_gb300 import build
    build.build()
    from sinkhorn_mixing_gb300 import binding
    return binding.lib()


def fake(i, off=0):
    return ctypes.c_void_p(A + i * GAP + off)


NULL = ctypes.c_void_p(0)


def pointers(order, change):
    p = {k: fake(i) for i, k in enumerate(order)}
    p.update(change)
    return [p[k] for k in order]


def norm(L, rows=4, d=64, dtype=BF16, center=0, eps=1e-6, **change):
    return L.hc_norm(rows, d, dtype, center, eps, *pointers(("x", "w", "b", "y"), change), None)


def norm_bwd(L, rows=4096, d=64, dtype=BF16, center=0, eps=1e-6, wsb=None, **change):
    p = pointers(("dy", "x", "w", "dx", "dw", "db", "ws"), change)
    wsb = L.hc_norm_backward_bytes(4096, 64, BF16) if wsb is None else wsb
    return L.hc_norm_backward(rows, d, dtype, center, eps, *p, wsb, None)


def embed(L, n=4, hc=4, d=64, vocab=100, size=8, dtype=BF16, scale=1.0, **change):
    return L.hc_embed(n, hc, d, vocab, size, dtype, scale,
                      *pointers(("ids", "table", "x"), change), None)


def embed_bwd(L, n=4, hc=4, d=64, vocab=100, size=8, dtype=BF16, scale=1.0, acc=0, wsb=None,
              **change):
    p = pointers(("ids", "dx", "dt", "ws"), change)
    wsb = L.hc_embed_backward_bytes(4, 64, 100) if wsb is None else wsb
    return L.hc_embed_backward(n, hc, d, vocab, size, dtype, scale, acc, *p, wsb, None)


def test_rows(L):
    for fn in (norm, norm_bwd):
        assert fn(L, rows=-1) == INVALID
        assert fn(L, d=0) == INVALID
        assert fn(L, d=20) == MISALIGNED
        assert fn(L, d=1 << 25) == UNSUPPORTED
        assert fn(L, rows=1 << 56) == UNSUPPORTED
        for dtype in (-1, 3):
            assert fn(L, dtype=dtype) == UNSUPPORTED
        for eps in (-1.0, math.nan, math.inf):
            assert fn(L, eps=eps) == INVALID


def test_norm(L):
    for k in ("x", "y"):
        assert norm(L, **{k: NULL}) == INVALID
        assert norm(L, **{k: fake(20, 8)}) == MISALIGNED
    for k in ("w", "b"):
        assert norm(L, **{k: fake(20, 4)}) == MISALIGNED
    assert norm(L, y=fake(0, 16)) == INVALID           # partly on x
    assert norm(L, y=fake(1)) == INVALID               # on the weight
    assert norm(L, b=fake(3, 496)) == INVALID
    assert norm(L, rows=0, x=NULL, y=NULL) == OK
    # 4 x 64 numbers of 2 bytes end at 512, of 4 bytes at 1024
    assert norm(L, dtype=F32, y=fake(0, 512)) == INVALID
    if no_gpu():
        assert norm(L, y=fake(0)) == CUDA              # in place
        assert norm(L, y=fake(0, 512)) == CUDA
        assert norm(L, w=NULL, b=NULL, center=1) == CUDA


def test_norm_backward(L):
    need = L.hc_norm_backward_bytes(4096, 64, BF16)
    assert need > 0 and L.hc_norm_backward_bytes(0, 64, BF16) == 0
    assert L.hc_norm_backward_bytes(4096, 12, BF16) == 0 == L.hc_norm_backward_bytes(4096, 64, 3)
    # wide rows need no more than their share, few rows none
    assert L.hc_norm_backward_bytes(1 << 20, 1 << 24, F32) < 1 << 36
    for dtype in (BF16, F16, F32):
        assert L.hc_norm_backward_bytes(2, 5120, dtype) == 0
        assert L.hc_norm_backward_bytes(20, 5120, dtype) > 0
        assert L.hc_norm_backward_bytes(1, 65536, dtype) > 0
    if no_gpu():
        assert norm_bwd(L, rows=2, ws=NULL, wsb=0) == CUDA
        assert norm_bwd(L, rows=2, ws=fake(0, 8)) == CUDA
    for k in ("dy", "x", "dx", "ws"):
        assert norm_bwd(L, **{k: NULL}) == INVALID
    for k in ("dy", "x", "w", "dx", "dw", "db"):
        assert norm_bwd(L, **{k: fake(20, 8)}) == MISALIGNED
    assert norm_bwd(L, ws=fake(20, 16)) == MISALIGNED
    assert norm_bwd(L, wsb=need - 1) == INVALID
    assert norm_bwd(L, dx=fake(0, 16)) == INVALID      # partly on dy
    assert norm_bwd(L, dx=fake(1)) == INVALID          # on x
    for k in ("dw", "db", "ws"):
        for on in range(4):
            assert norm_bwd(L, **{k: fake(on)}) == INVALID
    assert norm_bwd(L, dw=fake(5)) == INVALID          # on dbias
    if no_gpu():
        assert norm_bwd(L, dx=fake(0)) == CUDA         # in place
        assert norm_bwd(L, w=NULL, dw=NULL, db=NULL) == CUDA
    # no rows: only the parameters' gradients count
    assert norm_bwd(L, rows=0, dw=fake(5)) == INVALID
    assert norm_bwd(L, rows=0, dw=NULL, db=NULL, dx=NULL, ws=NULL) == OK


def test_embed(L):
    for fn in (embed, embed_bwd):
        assert fn(L, n=-1) == INVALID
        assert fn(L, vocab=0) == INVALID
        assert fn(L, d=12) == MISALIGNED
        for hc in (0, 2, 3, 16):
            assert fn(L, hc=hc) == UNSUPPORTED
        for size in (0, 2, 16):
            assert fn(L, size=size) == UNSUPPORTED
        assert fn(L, dtype=3) == UNSUPPORTED
        assert fn(L, vocab=(1 << 31) - 1) == UNSUPPORTED
        assert fn(L, n=(1 << 30) + 1) == UNSUPPORTED
        for scale in (math.nan, math.inf, -math.inf):
            assert fn(L, scale=scale) == INVALID
        assert fn(L, ids=NULL) == INVALID
        assert fn(L, ids=fake(20, 4)) == MISALIGNED
        assert fn(L, size=4, ids=fake(20, 2)) == MISALIGNED
    for k in ("table", "x"):
        assert embed(L, **{k: NULL}) == INVALID
        assert embed(L, **{k: fake(20, 8)}) == MISALIGNED
    assert embed(L, x=fake(0)) == INVALID
    assert embed(L, x=fake(1, 12784)) == INVALID
    assert embed(L, n=0, ids=NULL, x=NULL) == OK
    if no_gpu():
        assert embed(L, x=fake(1, 12800)) == CUDA      # behind 100 rows of 128 bytes
        assert embed(L, size=4, ids=fake(20, 4)) == CUDA


def test_embed_backward(L):
    need = L.hc_embed_backward_bytes(4, 64, 100)
    assert need > 0 and L.hc_embed_backward_bytes(0, 64, 100) == 0
    assert L.hc_embed_backward_bytes(4, 12, 100) == 0 == L.hc_embed_backward_bytes(4, 64, 0)
    for k in ("dx", "dt", "ws"):
        assert embed_bwd(L, **{k: NULL}) == INVALID
        assert embed_bwd(L, **{k: fake(20, 8)}) == MISALIGNED
    assert embed_bwd(L, wsb=need - 1) == INVALID
    assert embed_bwd(L, ws=fake(20, 128)) == MISALIGNED
    for on in (0, 1):
        assert embed_bwd(L, dt=fake(on)) == INVALID
        assert embed_bwd(L, ws=fake(on)) == INVALID
    assert embed_bwd(L, ws=fake(2)) == INVALID
    assert embed_bwd(L, n=0, dt=NULL) == INVALID
    if no_gpu():
        for acc in (0, 1):
            assert embed_bwd(L, acc=acc) == CUDA


def test_binding_refusals_without_a_gpu():
    import torch
    import sinkhorn_mixing_gb300 as hc
    x = torch.zeros(4, 64)
    ids = torch.zeros(4, dtype=torch.int64)
    for bad, what in ((x, ValueError), (x.double(), TypeError), (None, TypeError)):
        with pytest.raises(what):
            hc.hc_norm(bad)
        with pytest.raises(what):
            hc.hc_norm_backward(bad, bad)
    with pytest.raises(ValueError):
        hc.hc_embed(ids, x)                            # not on a GPU
    with pytest.raises(TypeError):
        hc.hc_embed(ids.float(), x)
    with pytest.raises(TypeError):
        hc.hc_embed_backward(x, ids.short(), 100)
