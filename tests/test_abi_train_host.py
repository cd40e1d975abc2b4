"""Refusals of the training entry points on the host: bad arguments return the documented status
before any CUDA call (the device pointers are fake addresses that nothing dereferences)."""
import ctypes
import math
import shutil

import os
import pytest

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA = 0, 1, 2, 3, 4
A, GAP = 1 << 20, 1 << 40

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


def _no_gpu():
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


def call(fn, order, scalars, **change):
    """fn(*scalars, pointers named in `order` at fake addresses, NULL stream), some changed."""
    p = {k: fake(i) for i, k in enumerate(order)}
    p.update(change)
    return fn(*scalars, *[p[k] for k in order], None)


CK = ("x", "codes", "scales")
PR = ("codes", "scales", "pre", "y")
PC = ("out", "residual", "post", "comb", "y", "codes", "scales")
PB = ("dy", "out", "osc", "res", "rsc", "post", "comb", "dout", "dpost", "dcomb", "dres")
MB = ("dy", "x", "xsc", "mixes", "w", "scale", "base", "dpost", "dcomb", "ds", "dx", "dw", "dsc",
      "db")


def mb(L, n=4, hc=4, d=64, iters=20, eps=1e-6, norm_eps=1e-20, ws=None, wsb=None, **change):
    p = {k: fake(i) for i, k in enumerate(MB)}
    p.update(change)
    need = L.hc_mixes_pre_backward_bytes(4, 4, 64)
    return L.hc_mixes_pre_backward(n, hc, d, iters, eps, norm_eps, *[p[k] for k in MB],
                                   fake(40) if ws is None else ws, need if wsb is None else wsb,
                                   None)


def test_rows(L):
    for fn in (L.hc_checkpoint, L.hc_restore):
        assert call(fn, CK, (-1, 64)) == INVALID
        assert call(fn, CK, (4, 0)) == INVALID
        assert call(fn, CK, (4, 12)) == MISALIGNED
        assert call(fn, CK, (1 << 56, 64)) == UNSUPPORTED
        assert call(fn, CK, (4, 1 << 25)) == UNSUPPORTED
        assert fn(0, 64, None, None, None, None) == OK
        assert call(fn, CK, (4, 64), codes=NULL) == INVALID
    for fn, order in ((L.hc_checkpoint, CK), (L.hc_restore, ("codes", "scales", "x"))):
        for k in ("x", "codes"):
            assert call(fn, order, (4, 64), **{k: fake(9, 8)}) == MISALIGNED
        for k in order:
            assert call(fn, order, (4, 64), **{k: NULL}) == INVALID
        if _no_gpu():
            assert call(fn, order, (4, 64), scales=fake(9, 3)) == CUDA   # any address
    # outputs on inputs and on each other
    assert call(L.hc_checkpoint, CK, (4, 64), codes=fake(0, 256)) == INVALID
    assert call(L.hc_checkpoint, CK, (4, 64), scales=fake(1, 240)) == INVALID
    assert call(L.hc_restore, CK, (4, 64), scales=fake(0, 128)) == INVALID


def test_pre_restore_and_post_checkpoint(L):
    assert call(L.hc_pre_restore, PR, (4, 3, 64)) == UNSUPPORTED
    assert call(L.hc_pre_restore, PR, (4, 4, 20)) == MISALIGNED
    assert call(L.hc_pre_restore, PR, (4, 4, 64), y=fake(2)) == INVALID
    assert call(L.hc_pre_restore, PR, (4, 4, 64), pre=NULL) == INVALID
    assert L.hc_pre_restore(0, 4, 64, None, None, None, None, None) == OK
    assert call(L.hc_post_checkpoint, PC, (4, 5, 64)) == UNSUPPORTED
    assert call(L.hc_post_checkpoint, PC, (1 << 40, 8, 1 << 24)) == UNSUPPORTED
    assert call(L.hc_post_checkpoint, PC, (4, 4, 64), y=fake(1, 16)) == INVALID
    assert call(L.hc_post_checkpoint, PC, (4, 4, 64), codes=fake(1)) == INVALID
    # in place is allowed for y, but not for the codes
    assert call(L.hc_post_checkpoint, PC, (4, 4, 64), y=fake(1), codes=fake(1, 512)) == INVALID
    if _no_gpu():
        assert call(L.hc_post_checkpoint, PC, (4, 4, 64), y=fake(1)) == CUDA


def test_post_backward(L):
    assert call(L.hc_post_backward, PB, (4, 2, 64)) == UNSUPPORTED
    assert call(L.hc_post_backward, PB, (-4, 4, 64)) == INVALID
    for k in ("dy", "out", "res", "post", "comb", "dout", "dpost", "dcomb"):
        assert call(L.hc_post_backward, PB, (4, 4, 64), **{k: NULL}) == INVALID
        assert call(L.hc_post_backward, PB, (4, 4, 64), **{k: fake(30, 8)}) == MISALIGNED
    assert call(L.hc_post_backward, PB, (4, 4, 64), dres=fake(30, 8)) == MISALIGNED
    assert call(L.hc_post_backward, PB, (4, 4, 64), dout=fake(0, 512)) == INVALID
    assert call(L.hc_post_backward, PB, (4, 4, 64), dres=fake(0, 16)) == INVALID
    assert call(L.hc_post_backward, PB, (4, 4, 64), dres=fake(3)) == INVALID
    assert call(L.hc_post_backward, PB, (4, 4, 64), dcomb=fake(6)) == INVALID
    # codes are half as long as bf16 rows: what lies behind them is free
    if _no_gpu():
        for change in (dict(dres=fake(0)), dict(dres=NULL), dict(osc=NULL, rsc=NULL),
                       dict(dout=fake(3, 1024))):
            assert call(L.hc_post_backward, PB, (4, 4, 64), **change) == CUDA
    assert call(L.hc_post_backward, PB, (4, 4, 64), rsc=NULL, dout=fake(3, 1024)) == INVALID


def test_mixes_pre_backward(L):
    need = L.hc_mixes_pre_backward_bytes(4, 4, 64)
    assert need > 0 and L.hc_mixes_pre_backward_bytes(0, 4, 64) == 0
    assert L.hc_mixes_pre_backward_bytes(4, 3, 64) == 0
    assert mb(L, hc=3) == UNSUPPORTED
    assert mb(L, d=12) == MISALIGNED
    assert mb(L, iters=0) == INVALID
    assert mb(L, iters=257) == UNSUPPORTED
    for bad in (-1.0, math.nan, math.inf):
        assert mb(L, eps=bad) == INVALID
        assert mb(L, norm_eps=bad) == INVALID
    for k in ("dy", "x", "mixes", "w", "scale", "base", "dpost", "dcomb", "dx", "dw", "dsc", "db"):
        assert mb(L, **{k: NULL}) == INVALID
        assert mb(L, **{k: fake(30, 4)}) == MISALIGNED
    assert mb(L, ds=fake(30, 4)) == MISALIGNED
    assert mb(L, ws=NULL) == INVALID
    assert mb(L, wsb=need - 1) == INVALID
    assert mb(L, ws=fake(40, 16)) == MISALIGNED
    assert mb(L, ws=fake(10)) == INVALID           # on dx
    assert mb(L, ws=fake(9)) == INVALID            # on dstream
    assert mb(L, dx=fake(9, 16)) == INVALID        # partly on dstream
    assert mb(L, dx=fake(1)) == INVALID            # on x
    assert mb(L, dw=fake(9)) == INVALID
    if _no_gpu():
        assert mb(L, dx=fake(9)) == CUDA           # dstream itself
        assert mb(L, ds=NULL) == CUDA
        assert mb(L, xsc=NULL) == CUDA
    # no tokens: the sums are still written, so their pointers count
    assert mb(L, n=0, dw=NULL) == INVALID
    assert mb(L, n=0, db=fake(11)) == INVALID


def test_binding_refusals_without_a_gpu():
    import torch
    import sinkhorn_mixing_gb300 as hc
    x = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hc.hc_checkpoint(x)                         # not on a GPU
    with pytest.raises(TypeError):
        hc.hc_checkpoint(x.float())
    with pytest.raises(TypeError):
        hc.hc_restore(x, x)
    with pytest.raises(TypeError):
        hc.hc_mixes_pre_backward(x.float(), x, None, None, None, None, None, None)
