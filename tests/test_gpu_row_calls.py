"""How hc_norm, hc_embed and their gradients are called: without launch overlap, for the first time
inside a capture, from several threads, and after a call that CUDA refuses (GPU)."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def hc():
    import sinkhorn_mixing_gb300 as lib
    lib.lib()
    yield lib
    assert lib.hc_device_error(clear=True) == 0


def inputs(n=500, d=1000, vocab=300, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    ids = torch.randint(-1, vocab, (n,), generator=g)
    c = dict(x=r(n, d).to(BF16), dy=r(n, d).to(BF16), w=r(d), b=r(d), ids=ids,
             table=r(vocab, d), dx=r(n, 4, d).to(BF16))
    return {k: v.cuda() for k, v in c.items()}


def calls(hc, c, **stream):
    """Every call's results; outputs and workspaces are the calls' own."""
    out = []
    for center in (False, True):
        out.append(hc.hc_norm(c["x"], c["w"], c["b"], eps=1e-5, center=center, **stream))
        out += hc.hc_norm_backward(c["dy"], c["x"], c["w"], eps=1e-5, center=center,
                                   want_dbias=True, **stream)
    out.append(hc.hc_embed(c["ids"], c["table"], scale=1.5, **stream))
    out.append(hc.hc_embed_backward(c["dx"], c["ids"], c["table"].shape[0], scale=1.5, **stream))
    return out


@pytest.mark.parametrize("n,d", [(500, 1000), (6000, 128), (40, 32776)])
def test_without_launch_overlap(hc, monkeypatch, n, d):
    c = inputs(n, d)
    want = calls(hc, c)
    monkeypatch.setenv("HCMIX_PDL", "0")
    for a, b in zip(calls(hc, c), want):
        assert torch.equal(a, b)


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured: what a kernel needs set up is set up there."""
    code = (
        "import sys; sys.path[:0] = [%r, %r]\n"
        "import torch, sinkhorn_mixing_gb300 as hc, test_gpu_row_calls as t\n"
        "c = t.inputs()\n"
        "torch.cuda.synchronize()\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    got = t.calls(hc, c)\n"
        "g.replay()\n"
        "torch.cuda.synchronize()\n"
        "assert all(torch.equal(a, b) for a, b in zip(got, t.calls(hc, c)))\n"
        "print('same')\n" % (ROOT, os.path.join(ROOT, "tests")))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_threads_and_streams(hc):
    """Four threads at once, each on a stream of its own and with its own outputs."""
    cs = [inputs(400 + 37 * i, 256 + 8 * i, 100, i) for i in range(4)]
    want = [calls(hc, c) for c in cs]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(10):
                got[i] = calls(hc, cs[i], stream=s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001 - reported below, in the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)


def test_a_call_that_cuda_refuses_leaves_no_error(hc):
    """The legacy default stream takes no work while a stream that synchronises with it is being
    captured; the next call does not see that error."""
    c = inputs(40, 64, 20)
    outs = dict(y=torch.empty_like(c["x"]), dx=torch.empty_like(c["x"]),
                dw=torch.empty_like(c["w"]), s=torch.empty_like(c["dx"]),
                dt=torch.empty_like(c["table"]),
                ws=torch.empty(max(hc.hc_norm_backward_bytes(40, 64),
                                   hc.hc_embed_backward_bytes(40, 64, 20)), dtype=torch.uint8,
                               device="cuda"))
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    fns = dict(
        norm=lambda: hc.hc_norm(c["x"], c["w"], y=outs["y"]),
        norm_backward=lambda: hc.hc_norm_backward(c["dy"], c["x"], c["w"], dx=outs["dx"],
                                                  dweight=outs["dw"], workspace=outs["ws"]),
        embed=lambda: hc.hc_embed(c["ids"], c["table"], x=outs["s"]),
        embed_backward=lambda: hc.hc_embed_backward(c["dx"], c["ids"], 20, dtable=outs["dt"],
                                                    workspace=outs["ws"]),
        no_rows=lambda: hc.hc_norm_backward(c["dy"][:0], c["x"][:0], c["w"], dx=c["x"][:0],
                                            dweight=outs["dw"], workspace=none),
        no_tokens=lambda: hc.hc_embed_backward(c["dx"][:0], c["ids"][:0], 20, dtable=outs["dt"],
                                               workspace=none))
    for fn in fns.values():
        fn()
    torch.cuda.synchronize()
    cuda = ctypes.CDLL("libcuda.so.1")
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert cuda.cuStreamCreate(ctypes.byref(stream), 0) == 0       # synchronises with the default
    try:
        for refused in fns:
            for after in fns:
                assert cuda.cuStreamBeginCapture_v2(stream, 2) == 0    # relaxed
                try:
                    with pytest.raises(hc.HcError, match="HC_ERR_CUDA"):
                        fns[refused]()
                finally:
                    status = cuda.cuStreamEndCapture(stream, ctypes.byref(graph))
                assert status == 901, status                           # capture invalidated
                fns[after]()
                torch.cuda.synchronize()
    finally:
        assert cuda.cuStreamDestroy_v2(stream) == 0
