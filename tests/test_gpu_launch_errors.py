"""A call that CUDA refuses leaves nothing behind for the next one (GPU).

The refusal is CUDA's own, on the host: the legacy default stream takes no work while a stream that
synchronises with it is being captured.
"""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hc():
    import sinkhorn_mixing_gb300 as lib
    lib.lib()
    return lib


def calls(hc):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(40, 4, 64, generator=g).to(torch.bfloat16).cuda()
    out = torch.randn(40, 64, generator=g).to(torch.bfloat16).cuda()
    post, comb = torch.rand(40, 4, generator=g).cuda(), torch.rand(40, 4, 4, generator=g).cuda()
    mixes = torch.randn(40, 24, generator=g).cuda()
    w, s, b = torch.randn(24, 256, generator=g).cuda(), torch.ones(3).cuda(), torch.zeros(24).cuda()
    codes, scales = hc.hc_checkpoint(x)
    y, y1 = torch.empty_like(x), torch.empty_like(out)
    pre, split = torch.empty_like(post), (torch.empty_like(post), torch.empty_like(comb))
    outs = dict(dx=torch.empty_like(x), dw_mix=torch.empty_like(w), dscale=torch.empty_like(s),
                dbase=torch.empty_like(b),
                workspace=torch.empty(hc.hc_mixes_pre_backward_bytes(40, 4, 64), dtype=torch.uint8,
                                      device="cuda"))
    none = dict(outs, dx=x[:0], workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    return dict(
        checkpoint=lambda: hc.hc_checkpoint(x, codes=codes, scales=scales),
        restore=lambda: hc.hc_restore(codes, scales, x=y),
        pre=lambda: hc.hc_pre(x, post, y=y1),
        post=lambda: hc.hc_post(out, x, post, comb, y=y),
        split=lambda: hc.hc_split_sinkhorn(mixes, s, b, pre=pre, post=split[0], comb=split[1]),
        backward=lambda: hc.hc_mixes_pre_backward(out, x, mixes, w, s, b, post, comb, **outs),
        no_tokens=lambda: hc.hc_mixes_pre_backward(out[:0], x[:0], mixes[:0], w, s, b, post[:0],
                                                   comb[:0], **none))


@pytest.mark.parametrize("refused", ["checkpoint", "post", "backward", "no_tokens"])
def test_refused_call_leaves_no_error(hc, refused):
    fns = calls(hc)
    for fn in fns.values():
        fn()
    torch.cuda.synchronize()
    cuda = ctypes.CDLL("libcuda.so.1")
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert cuda.cuStreamCreate(ctypes.byref(stream), 0) == 0       # synchronises with the default
    try:
        for after in fns:
            assert cuda.cuStreamBeginCapture_v2(stream, 2) == 0    # relaxed
            try:
                with pytest.raises(hc.HcError, match="HC_ERR_CUDA"):
                    fns[refused]()
            finally:
                status = cuda.cuStreamEndCapture(stream, ctypes.byref(graph))
            assert status == 901, status                           # capture invalidated
            before = hc.hc_launch_count()
            fns[after]()
            assert after == "no_tokens" or hc.hc_launch_count() > before
            torch.cuda.synchronize()
    finally:
        assert cuda.cuStreamDestroy_v2(stream) == 0
