"""Thin Python binding of libhcmix.so (argument marshalling only).

Every function has the name of the C entry point it calls and does nothing
but check tensor dtypes/devices/contiguity, allocate missing outputs with
torch (as the reference wrapper does with ``new_empty``), and pass raw device
pointers plus the current CUDA stream.  All arithmetic runs in the library's
kernels; there is no fallback path: if the library is missing or a call
fails, an exception is raised.

Leading dimensions are flattened to the token count n, as the pages' wrapper
views ``[b, s, ...]`` tensors as ``[n, ...]``; outputs keep the caller's
leading dimensions.
"""
import ctypes
import functools
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhcmix.so")

HC_OK = 0
_lib = None


class HcError(RuntimeError):
    """A non-OK hc_status returned by the library."""

    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s: %s" % (what, status_string(status)))


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libhcmix.so is not built (%s); run `python -m "
                "sinkhorn_mixing_gb300.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        L.hc_status_string.argtypes = [i32]
        L.hc_status_string.restype = ctypes.c_char_p
        L.hc_abi_version.restype = i32
        L.hc_mixes.argtypes = [i64, i32, i64, f32, P, P, P, P]
        L.hc_split_sinkhorn.argtypes = [i64, i32, i32, f32, P, P, P, P, P, P, P]
        L.hc_pre.argtypes = [i64, i32, i64, P, P, P, P]
        L.hc_post.argtypes = [i64, i32, i64, P, P, P, P, P, P]
        L.hc_mixes_pre.argtypes = [i64, i32, i64, i32, f32, f32, P, P, P, P, P, P, P, P, P, P,
                                   ctypes.c_size_t, P]
        L.hc_mixes_pre_norm.argtypes = [i64, i32, i64, i32, f32, f32, P, P, P, P, P, f32, P, P,
                                        P, P, P, P, ctypes.c_size_t, P]
        L.hc_post_mixes_pre.argtypes = [i64, i32, i64, P, P, P, P, P, i32, f32, f32, P, P, P, P,
                                        P, P, P, P, P, ctypes.c_size_t, P]
        L.hc_checkpoint.argtypes = [i64, i64, P, P, P, P]
        L.hc_restore.argtypes = [i64, i64, P, P, P, P]
        L.hc_pre_restore.argtypes = [i64, i32, i64, P, P, P, P, P]
        L.hc_post_checkpoint.argtypes = [i64, i32, i64, P, P, P, P, P, P, P, P]
        L.hc_post_backward.argtypes = [i64, i32, i64, P, P, P, P, P, P, P, P, P, P, P, P]
        L.hc_mixes_pre_backward.argtypes = [i64, i32, i64, i32, f32, f32, P, P, P, P, P, P, P, P,
                                            P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.hc_mixes_pre_backward_bytes.argtypes = [i64, i32, i64]
        L.hc_mixes_pre_backward_bytes.restype = ctypes.c_size_t
        L.hc_norm.argtypes = [i64, i64, i32, i32, f32, P, P, P, P, P]
        L.hc_norm_backward.argtypes = [i64, i64, i32, i32, f32, P, P, P, P, P, P, P,
                                       ctypes.c_size_t, P]
        L.hc_norm_backward_bytes.argtypes = [i64, i64, i32]
        L.hc_norm_backward_bytes.restype = ctypes.c_size_t
        L.hc_embed.argtypes = [i64, i32, i64, i64, i32, i32, f32, P, P, P, P]
        L.hc_embed_backward.argtypes = [i64, i32, i64, i64, i32, i32, f32, i32, P, P, P, P,
                                        ctypes.c_size_t, P]
        L.hc_embed_backward_bytes.argtypes = [i64, i64, i64]
        L.hc_embed_backward_bytes.restype = ctypes.c_size_t
        L.hc_workspace_bytes.argtypes = [i64, i32, i64]
        L.hc_workspace_bytes.restype = ctypes.c_size_t
        L.hc_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint), i32]
        L.hc_launch_count.restype = ctypes.c_uint64
        L.hc_selftest_wait_timeout.argtypes = [ctypes.c_uint64, P]
        L.hc_selftest_wait_timeout.restype = i32
        for f in ("hc_mixes", "hc_split_sinkhorn", "hc_pre", "hc_post", "hc_mixes_pre",
                  "hc_mixes_pre_norm", "hc_post_mixes_pre", "hc_device_error", "hc_checkpoint",
                  "hc_restore", "hc_pre_restore", "hc_post_checkpoint", "hc_post_backward",
                  "hc_mixes_pre_backward", "hc_norm", "hc_norm_backward", "hc_embed",
                  "hc_embed_backward"):
            getattr(L, f).restype = i32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().hc_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != HC_OK:
        raise HcError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    # a plain int (or None for NULL): ctypes converts it for c_void_p arguments
    return None if t is None else t.data_ptr()


# The raw handle of the current stream without building a Stream object
# (a few microseconds per call on the decode path); public API otherwise.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev: torch.device, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _call(dev: torch.device, fn, *args):
    """fn(*args) with `dev` as the current device, switching (and back) only
    when it is not already current."""
    cur = torch.cuda.current_device()
    if cur == dev.index:
        return fn(*args)
    torch.cuda.set_device(dev.index)
    try:
        return fn(*args)
    finally:
        torch.cuda.set_device(cur)


def _need(t: torch.Tensor, name: str, dtype, dev=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dev is not None and t.get_device() != dev.index:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _out(t, name, shape, dtype, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _need(t, name, dtype, dev)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t


def _stream_dims(x: torch.Tensor):
    if x.dim() < 2:
        raise ValueError("x must be [..., hc, d]")
    lead = tuple(x.shape[:-2])
    hc, d = int(x.shape[-2]), int(x.shape[-1])
    n = 1
    for s in lead:
        n *= int(s)
    return lead, n, hc, d


def abi_version() -> int:
    return int(lib().hc_abi_version())


@functools.lru_cache(maxsize=256)
def hc_workspace_bytes(n: int, hc: int, d: int) -> int:
    # a pure function of its arguments (hcmix.h), so it is asked once per shape
    return int(lib().hc_workspace_bytes(int(n), int(hc), int(d)))


def hc_mixes(x, w_mix, norm_eps: float = 1e-20, mixes=None, stream=None):
    """x [..., hc, d] bf16, w_mix [(2+hc)*hc, hc*d] fp32 -> mixes [..., mix_hc] fp32."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    lead, n, hc, d = _stream_dims(x)
    _need(w_mix, "w_mix", torch.float32, dev)
    mix = (2 + hc) * hc
    mixes = _out(mixes, "mixes", lead + (mix,), torch.float32, dev)
    _check(_call(dev, lib().hc_mixes, n, hc, d, float(norm_eps), _ptr(x), _ptr(w_mix),
                 _ptr(mixes), _stream(dev, stream)), "hc_mixes")
    return mixes


def hc_split_sinkhorn(mixes, hc_scale, hc_base, hc_mult: int = 4, sinkhorn_iters: int = 20,
                      eps: float = 1e-6, pre=None, post=None, comb=None, stream=None):
    """mixes [..., (2+hc)*hc] fp32 -> pre [..., hc], post [..., hc], comb [..., hc, hc]."""
    _need(mixes, "mixes", torch.float32)
    dev = mixes.device
    hc = int(hc_mult)
    mix = (2 + hc) * hc
    if mixes.shape[-1] != mix:
        raise ValueError("mixes last dim must be %d" % mix)
    lead = tuple(mixes.shape[:-1])
    n = mixes.numel() // mix
    _need(hc_scale, "hc_scale", torch.float32, dev)
    _need(hc_base, "hc_base", torch.float32, dev)
    pre = _out(pre, "pre", lead + (hc,), torch.float32, dev)
    post = _out(post, "post", lead + (hc,), torch.float32, dev)
    comb = _out(comb, "comb", lead + (hc, hc), torch.float32, dev)
    _check(_call(dev, lib().hc_split_sinkhorn, n, hc, int(sinkhorn_iters), float(eps),
                 _ptr(mixes), _ptr(hc_scale), _ptr(hc_base), _ptr(pre), _ptr(post), _ptr(comb),
                 _stream(dev, stream)), "hc_split_sinkhorn")
    return pre, post, comb


def hc_pre(x, pre, y=None, stream=None):
    """x [..., hc, d] bf16, pre [..., hc] fp32 -> y [..., d] bf16."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    lead, n, hc, d = _stream_dims(x)
    _need(pre, "pre", torch.float32, dev)
    if pre.numel() != n * hc:
        raise ValueError("pre must hold n*hc values")
    y = _out(y, "y", lead + (d,), torch.bfloat16, dev)
    _check(_call(dev, lib().hc_pre, n, hc, d, _ptr(x), _ptr(pre), _ptr(y), _stream(dev, stream)),
           "hc_pre")
    return y


def hc_post(out, residual, post, comb, y=None, stream=None):
    """out [..., d] bf16, residual [..., hc, d] bf16, post [..., hc], comb [..., hc, hc]
    -> y [..., hc, d] bf16 (y may be residual itself)."""
    _need(residual, "residual", torch.bfloat16)
    dev = residual.device
    lead, n, hc, d = _stream_dims(residual)
    _need(out, "out", torch.bfloat16, dev)
    if out.numel() != n * d:
        raise ValueError("out must hold n*d values")
    _need(post, "post", torch.float32, dev)
    _need(comb, "comb", torch.float32, dev)
    if post.numel() != n * hc or comb.numel() != n * hc * hc:
        raise ValueError("post/comb sizes do not match residual")
    y = _out(y, "y", lead + (hc, d), torch.bfloat16, dev)
    _check(_call(dev, lib().hc_post, n, hc, d, _ptr(out), _ptr(residual), _ptr(post), _ptr(comb),
                 _ptr(y), _stream(dev, stream)), "hc_post")
    return y


def hc_mixes_pre(x, w_mix, hc_scale, hc_base, sinkhorn_iters: int = 20, eps: float = 1e-6,
                 norm_eps: float = 1e-20, want_mixes: bool = False, mixes=None, pre=None,
                 post=None, comb=None, y=None, workspace=None, stream=None):
    """Fused mix projection + split/Sinkhorn + collapse.
    Returns (y, pre, post, comb, mixes-or-None)."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    lead, n, hc, d = _stream_dims(x)
    mix = (2 + hc) * hc
    _need(w_mix, "w_mix", torch.float32, dev)
    _need(hc_scale, "hc_scale", torch.float32, dev)
    _need(hc_base, "hc_base", torch.float32, dev)
    if want_mixes or mixes is not None:
        mixes = _out(mixes, "mixes", lead + (mix,), torch.float32, dev)
    pre = _out(pre, "pre", lead + (hc,), torch.float32, dev)
    post = _out(post, "post", lead + (hc,), torch.float32, dev)
    comb = _out(comb, "comb", lead + (hc, hc), torch.float32, dev)
    y = _out(y, "y", lead + (d,), torch.bfloat16, dev)
    wbytes = 0
    if mixes is None or hc == 8:
        # the mix numbers when not returned; at hc = 8 also W converted for
        # the tensor-core projection (hcmix.h, hc_workspace_bytes)
        wbytes = hc_workspace_bytes(n, hc, d)
        if workspace is None and wbytes:
            workspace = torch.empty(wbytes, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
        wbytes = workspace.numel()
    _check(_call(dev, lib().hc_mixes_pre, n, hc, d, int(sinkhorn_iters), float(eps),
                 float(norm_eps), _ptr(x), _ptr(w_mix), _ptr(hc_scale), _ptr(hc_base),
                 _ptr(mixes), _ptr(pre), _ptr(post), _ptr(comb), _ptr(y), _ptr(workspace), wbytes,
                 _stream(dev, stream)), "hc_mixes_pre")
    return y, pre, post, comb, mixes


def hc_mixes_pre_norm(x, w_mix, hc_scale, hc_base, rms_weight, sinkhorn_iters: int = 20,
                      eps: float = 1e-6, norm_eps: float = 1e-20, rms_eps: float = 1e-20,
                      want_mixes: bool = False, mixes=None, pre=None, post=None, comb=None, y=None,
                      workspace=None, stream=None):
    """hc_mixes_pre whose collapsed output y is also RMS-normalised with
    rms_weight [d].  Returns (y, pre, post, comb, mixes-or-None)."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    lead, n, hc, d = _stream_dims(x)
    mix = (2 + hc) * hc
    _need(w_mix, "w_mix", torch.float32, dev)
    _need(hc_scale, "hc_scale", torch.float32, dev)
    _need(hc_base, "hc_base", torch.float32, dev)
    _need(rms_weight, "rms_weight", torch.float32, dev)
    if tuple(rms_weight.shape) != (d,):
        raise ValueError("rms_weight must have shape (%d,)" % d)
    if want_mixes or mixes is not None:
        mixes = _out(mixes, "mixes", lead + (mix,), torch.float32, dev)
    pre = _out(pre, "pre", lead + (hc,), torch.float32, dev)
    post = _out(post, "post", lead + (hc,), torch.float32, dev)
    comb = _out(comb, "comb", lead + (hc, hc), torch.float32, dev)
    y = _out(y, "y", lead + (d,), torch.bfloat16, dev)
    wbytes = 0
    if mixes is None or hc == 8:
        wbytes = hc_workspace_bytes(n, hc, d)
        if workspace is None and wbytes:
            workspace = torch.empty(wbytes, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
        wbytes = workspace.numel()
    _check(_call(dev, lib().hc_mixes_pre_norm, n, hc, d, int(sinkhorn_iters), float(eps),
                 float(norm_eps), _ptr(x), _ptr(w_mix), _ptr(hc_scale), _ptr(hc_base),
                 _ptr(rms_weight), float(rms_eps), _ptr(mixes), _ptr(pre), _ptr(post), _ptr(comb),
                 _ptr(y), _ptr(workspace), wbytes, _stream(dev, stream)), "hc_mixes_pre_norm")
    return y, pre, post, comb, mixes


def hc_post_mixes_pre(out, residual, post, comb, w_mix, hc_scale, hc_base,
                      sinkhorn_iters: int = 20, eps: float = 1e-6, norm_eps: float = 1e-20,
                      x_next=None, want_mixes: bool = False, mixes=None, pre=None,
                      post_next=None, comb_next=None, y=None, workspace=None, stream=None):
    """hc_post of one sublayer and hc_mixes_pre of the next in one call:
    x_next = hc_post(out, residual, post, comb) (x_next may be residual), then
    the next sublayer's (y, pre, post, comb[, mixes]) from x_next with its
    parameters w_mix, hc_scale, hc_base.
    Returns (x_next, y, pre, post, comb, mixes-or-None)."""
    _need(residual, "residual", torch.bfloat16)
    dev = residual.device
    lead, n, hc, d = _stream_dims(residual)
    _need(out, "out", torch.bfloat16, dev)
    if out.numel() != n * d:
        raise ValueError("out must hold n*d values")
    _need(post, "post", torch.float32, dev)
    _need(comb, "comb", torch.float32, dev)
    if post.numel() != n * hc or comb.numel() != n * hc * hc:
        raise ValueError("post/comb sizes do not match residual")
    mix = (2 + hc) * hc
    _need(w_mix, "w_mix", torch.float32, dev)
    _need(hc_scale, "hc_scale", torch.float32, dev)
    _need(hc_base, "hc_base", torch.float32, dev)
    x_next = _out(x_next, "x_next", lead + (hc, d), torch.bfloat16, dev)
    if want_mixes or mixes is not None:
        mixes = _out(mixes, "mixes", lead + (mix,), torch.float32, dev)
    pre = _out(pre, "pre", lead + (hc,), torch.float32, dev)
    post_next = _out(post_next, "post_next", lead + (hc,), torch.float32, dev)
    comb_next = _out(comb_next, "comb_next", lead + (hc, hc), torch.float32, dev)
    y = _out(y, "y", lead + (d,), torch.bfloat16, dev)
    wbytes = 0
    if mixes is None or hc == 8:
        wbytes = hc_workspace_bytes(n, hc, d)
        if workspace is None and wbytes:
            workspace = torch.empty(wbytes, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
        wbytes = workspace.numel()
    _check(_call(dev, lib().hc_post_mixes_pre, n, hc, d, _ptr(out), _ptr(residual), _ptr(post),
                 _ptr(comb), _ptr(x_next), int(sinkhorn_iters), float(eps), float(norm_eps),
                 _ptr(w_mix), _ptr(hc_scale), _ptr(hc_base), _ptr(mixes), _ptr(pre),
                 _ptr(post_next), _ptr(comb_next), _ptr(y), _ptr(workspace), wbytes,
                 _stream(dev, stream)), "hc_post_mixes_pre")
    return x_next, y, pre, post_next, comb_next, mixes


KEPT_BLOCK = 32  # channels that share a scale byte (hcmix.h, hc_checkpoint)

# The functions below run once per sublayer on the host's time, which for small
# calls is most of theirs: shapes stay torch.Size, and each check is made once.
_BF16, _F32, _F8, _U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8


def _on(t, name, dtype, index):
    """_need on device `index`, in fewer steps."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index or \
            not t.is_contiguous():
        _need(t, name, dtype, torch.device("cuda", index))


def _sized(t, name, count, dtype, index):
    _on(t, name, dtype, index)
    if t.numel() != count:
        raise ValueError("%s must hold %d values, got %d" % (name, count, t.numel()))
    return t.data_ptr()


def _made(t, name, shape, dtype, dev, stream):
    """An output: the caller's, checked, or a new one.  One made for another stream
    is that stream's own memory, so that nothing the current stream has still to do
    can touch it, and it is not handed out again before the current stream, which
    may read it, is done with it either."""
    if t is None:
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=dev)
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=dev)
        t.record_stream(torch.cuda.current_stream(dev))
        return t
    _on(t, name, dtype, dev.index)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
    return t


def _kept(t, name, shape, index):
    """A kept tensor of `shape`, bf16 or (codes, scales): the pointers to its
    data and to its scales (None)."""
    if isinstance(t, torch.Tensor):
        _on(t, name, _BF16, index)
        if t.shape != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
        return t.data_ptr(), None
    if not isinstance(t, (tuple, list)) or len(t) != 2:
        raise TypeError("%s must be a bf16 tensor or (codes, scales)" % name)
    codes, scales = t
    _on(codes, name + " codes", _F8, index)
    _on(scales, name + " scales", _U8, index)
    if codes.shape != shape:
        raise ValueError("%s codes must have shape %s, got %s" % (name, shape, tuple(codes.shape)))
    want = shape[:-1] + ((shape[-1] + KEPT_BLOCK - 1) // KEPT_BLOCK,)
    if scales.shape != want:
        raise ValueError("%s scales must have shape %s, got %s" % (name, want,
                                                                   tuple(scales.shape)))
    return codes.data_ptr(), scales.data_ptr()


def _rows_of(t):
    shape = tuple(t.shape)
    if len(shape) < 1:
        raise ValueError("a row of channels at least is needed")
    d = shape[-1]
    n = 1
    for s in shape[:-1]:
        n *= s
    return shape, n, d


def _tokens_of(t):
    shape = tuple(t.shape)
    if len(shape) < 2:
        raise ValueError("a stream must be [..., hc, d]")
    n = 1
    for s in shape[:-2]:
        n *= s
    return shape, n, shape[-2], shape[-1]


_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(name, dev, stream, *args):
    """The C entry point `name` on dev's current (or the given) stream."""
    fn = getattr(_lib if _lib is not None else lib(), name)
    if stream is not None:
        raw = stream.cuda_stream
    elif _raw_stream is not None:
        raw = _raw_stream(dev.index)
    else:
        raw = torch.cuda.current_stream(dev).cuda_stream
    status = fn(*args, raw) if _get_device() == dev.index else _call(dev, fn, *args, raw)
    if status != HC_OK:
        raise HcError(status, name)


def hc_checkpoint(x, codes=None, scales=None, stream=None):
    """x [..., d] bf16 -> codes [..., d] float8_e4m3fn, scales [..., ceil(d / 32)]
    uint8: a channel's value is code * 2^(scale - 127)."""
    _need(x, "x", _BF16)
    dev = x.device
    shape, n, d = _rows_of(x)
    codes = _made(codes, "codes", shape, _F8, dev, stream)
    scales = _made(scales, "scales", shape[:-1] + ((d + KEPT_BLOCK - 1) // KEPT_BLOCK,), _U8, dev,
                   stream)
    _run("hc_checkpoint", dev, stream, n, d, x.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return codes, scales


def hc_restore(codes, scales, x=None, stream=None):
    """codes [..., d], scales [..., ceil(d / 32)] of hc_checkpoint -> x [..., d] bf16."""
    _need(codes, "codes", _F8)
    dev = codes.device
    shape, n, d = _rows_of(codes)
    cp, sp = _kept((codes, scales), "x", shape, dev.index)
    x = _made(x, "x", shape, _BF16, dev, stream)
    _run("hc_restore", dev, stream, n, d, cp, sp, x.data_ptr())
    return x


def hc_pre_restore(codes, scales, pre, y=None, stream=None):
    """hc_pre of a kept stream: codes [..., hc, d], scales, pre [..., hc] -> y [..., d] bf16."""
    _need(codes, "codes", _F8)
    dev = codes.device
    shape, n, hc, d = _tokens_of(codes)
    cp, sp = _kept((codes, scales), "x", shape, dev.index)
    pp = _sized(pre, "pre", n * hc, _F32, dev.index)
    y = _made(y, "y", shape[:-2] + (d,), _BF16, dev, stream)
    _run("hc_pre_restore", dev, stream, n, hc, d, cp, sp, pp, y.data_ptr())
    return y


def hc_post_checkpoint(out, residual, post, comb, y=None, codes=None, scales=None, stream=None):
    """hc_post that also keeps the new stream in 8 bits (y may be residual itself).
    Returns (y, codes, scales)."""
    _need(residual, "residual", _BF16)
    dev = residual.device
    shape, n, hc, d = _tokens_of(residual)
    op = _sized(out, "out", n * d, _BF16, dev.index)
    pp = _sized(post, "post", n * hc, _F32, dev.index)
    cb = _sized(comb, "comb", n * hc * hc, _F32, dev.index)
    y = _made(y, "y", shape, _BF16, dev, stream)
    codes = _made(codes, "codes", shape, _F8, dev, stream)
    scales = _made(scales, "scales", shape[:-1] + ((d + KEPT_BLOCK - 1) // KEPT_BLOCK,), _U8, dev,
                   stream)
    _run("hc_post_checkpoint", dev, stream, n, hc, d, op, residual.data_ptr(), pp, cb,
         y.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return y, codes, scales


def hc_post_backward(dy, out, residual, post, comb, want_dresidual: bool = False, dout=None,
                     dpost=None, dcomb=None, dresidual=None, stream=None):
    """Gradients of hc_post from dy [..., hc, d] bf16.  out [..., d] and residual
    [..., hc, d] are bf16 tensors or (codes, scales) of hc_checkpoint.
    Returns (dout, dpost, dcomb, dresidual-or-None); dresidual may be dy itself."""
    _need(dy, "dy", _BF16)
    dev = dy.device
    shape, n, hc, d = _tokens_of(dy)
    lead = shape[:-2]
    op, osp = _kept(out, "out", lead + (d,), dev.index)
    rp, rsp = _kept(residual, "residual", shape, dev.index)
    pp = _sized(post, "post", n * hc, _F32, dev.index)
    cb = _sized(comb, "comb", n * hc * hc, _F32, dev.index)
    dout = _made(dout, "dout", lead + (d,), _BF16, dev, stream)
    dpost = _made(dpost, "dpost", lead + (hc,), _F32, dev, stream)
    dcomb = _made(dcomb, "dcomb", lead + (hc, hc), _F32, dev, stream)
    if want_dresidual or dresidual is not None:
        dresidual = _made(dresidual, "dresidual", shape, _BF16, dev, stream)
    _run("hc_post_backward", dev, stream, n, hc, d, dy.data_ptr(), op, osp, rp, rsp, pp, cb,
         dout.data_ptr(), dpost.data_ptr(), dcomb.data_ptr(),
         None if dresidual is None else dresidual.data_ptr())
    return dout, dpost, dcomb, dresidual


@functools.lru_cache(maxsize=256)
def hc_mixes_pre_backward_bytes(n: int, hc: int, d: int) -> int:
    return int(lib().hc_mixes_pre_backward_bytes(int(n), int(hc), int(d)))


def hc_mixes_pre_backward(dy, x, mixes, w_mix, hc_scale, hc_base, dpost, dcomb, dstream=None,
                          sinkhorn_iters: int = 20, eps: float = 1e-6, norm_eps: float = 1e-20,
                          dx=None, dw_mix=None, dscale=None, dbase=None, workspace=None,
                          stream=None):
    """Gradients of hc_mixes_pre from dy [..., d] bf16, dpost [..., hc] and dcomb
    [..., hc, hc]; with dstream [..., hc, d] (the dy of hc_post_backward) also of the
    stream that hc_post carried past the sublayer.  x [..., hc, d] is a bf16 tensor or
    (codes, scales); mixes is what hc_mixes_pre returned.
    Returns (dx, dw_mix, dscale, dbase); dx may be dstream itself."""
    _need(dy, "dy", _BF16)
    dev = dy.device
    data = x[0] if isinstance(x, (tuple, list)) and x else x
    if not isinstance(data, torch.Tensor):
        raise TypeError("x must be a bf16 tensor or (codes, scales)")
    shape, n, hc, d = _tokens_of(data)
    xp, xsp = _kept(x, "x", shape, dev.index)
    mix, F = (2 + hc) * hc, hc * d
    if dy.shape != shape[:-2] + (d,):
        raise ValueError("dy must have shape %s, got %s" % (shape[:-2] + (d,), tuple(dy.shape)))
    mp = _sized(mixes, "mixes", n * mix, _F32, dev.index)
    wp = _sized(w_mix, "w_mix", mix * F, _F32, dev.index)
    sp = _sized(hc_scale, "hc_scale", 3, _F32, dev.index)
    bp = _sized(hc_base, "hc_base", mix, _F32, dev.index)
    pp = _sized(dpost, "dpost", n * hc, _F32, dev.index)
    cp = _sized(dcomb, "dcomb", n * hc * hc, _F32, dev.index)
    gp = None if dstream is None else _sized(dstream, "dstream", n * F, _BF16, dev.index)
    dx = _made(dx, "dx", shape, _BF16, dev, stream)
    dw_mix = _made(dw_mix, "dw_mix", (mix, F), _F32, dev, stream)
    dscale = _made(dscale, "dscale", (3,), _F32, dev, stream)
    dbase = _made(dbase, "dbase", (mix,), _F32, dev, stream)
    if workspace is None:
        workspace = _made(None, "workspace", (hc_mixes_pre_backward_bytes(n, hc, d),), _U8, dev,
                          stream)
    else:
        _need(workspace, "workspace", _U8, dev)
    _run("hc_mixes_pre_backward", dev, stream, n, hc, d, sinkhorn_iters, eps, norm_eps,
         dy.data_ptr(), xp, xsp, mp, wp, sp, bp, pp, cp, gp, dx.data_ptr(), dw_mix.data_ptr(),
         dscale.data_ptr(), dbase.data_ptr(), workspace.data_ptr(), workspace.numel())
    return dx, dw_mix, dscale, dbase


_ROW_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # hcmix.h, hc_dtype


def _row_type(dtype, name):
    code = _ROW_TYPES.get(dtype)
    if code is None:
        raise TypeError("%s must be bfloat16, float16 or float32, got %s" % (name, dtype))
    return code


def _row_tensor(t, name):
    """A tensor of rows [..., d]: its device, shape, rows, width, type and the type's code."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    dtype, shape = t.dtype, t.shape
    code = _row_type(dtype, name)
    if not (t.is_cuda and t.is_contiguous()):
        _need(t, name, dtype)
    if len(shape) < 1:
        raise ValueError("a row of channels at least is needed")
    d = shape[-1]
    return t.device, shape, t.numel() // d if d else 0, d, dtype, code


def hc_norm(x, weight=None, bias=None, eps: float = 1e-20, center: bool = False, y=None,
            stream=None):
    """x [..., d] bf16, fp16 or fp32 -> (x - mean) / sqrt(variance + eps) * weight + bias over
    each row, in x's type (y may be x itself).  center=False leaves the mean in and takes the
    mean square (RMS norm).  weight, bias [d] fp32, or None."""
    dev, shape, n, d, dtype, code = _row_tensor(x, "x")
    wp = None if weight is None else _sized(weight, "weight", d, _F32, dev.index)
    bp = None if bias is None else _sized(bias, "bias", d, _F32, dev.index)
    y = _made(y, "y", shape, dtype, dev, stream)
    _run("hc_norm", dev, stream, n, d, code, bool(center), eps, x.data_ptr(), wp, bp, y.data_ptr())
    return y


@functools.lru_cache(maxsize=256)
def hc_norm_backward_bytes(rows: int, d: int, dtype=torch.bfloat16) -> int:
    return int(lib().hc_norm_backward_bytes(int(rows), int(d), _row_type(dtype, "rows")))


def hc_norm_backward(dy, x, weight=None, eps: float = 1e-20, center: bool = False,
                     want_dweight: bool = True, want_dbias: bool = False, dx=None, dweight=None,
                     dbias=None, workspace=None, stream=None):
    """Gradients of hc_norm from dy [..., d], of x's type, and x, the forward call's input.
    Returns (dx, dweight-or-None, dbias-or-None); dx may be dy itself."""
    dev, shape, n, d, dtype, code = _row_tensor(x, "x")
    _on(dy, "dy", dtype, dev.index)
    if dy.shape != shape:
        raise ValueError("dy must have shape %s, got %s" % (tuple(shape), tuple(dy.shape)))
    wp = None if weight is None else _sized(weight, "weight", d, _F32, dev.index)
    dx = _made(dx, "dx", shape, dtype, dev, stream)
    if want_dweight or dweight is not None:
        dweight = _made(dweight, "dweight", (d,), _F32, dev, stream)
    if want_dbias or dbias is not None:
        dbias = _made(dbias, "dbias", (d,), _F32, dev, stream)
    if workspace is not None:
        _need(workspace, "workspace", _U8, dev)
    else:
        need = hc_norm_backward_bytes(n, d, dtype)   # 0 for few rows
        if need:
            workspace = _made(None, "workspace", (need,), _U8, dev, stream)
    _run("hc_norm_backward", dev, stream, n, d, code, bool(center), eps, dy.data_ptr(),
         x.data_ptr(), wp, dx.data_ptr(), _ptr(dweight), _ptr(dbias), _ptr(workspace),
         0 if workspace is None else workspace.numel())
    return dx, dweight, dbias


def _ids_of(ids):
    """Token ids, int32 or int64: their device, shape, count and bytes each."""
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be int32 or int64, got %s" % ids.dtype)
    _need(ids, "ids", ids.dtype)
    return ids.device, tuple(ids.shape), ids.numel(), ids.element_size()


def hc_embed(ids, table, hc_mult: int = 4, scale: float = 1.0, x=None, stream=None):
    """ids [...] int32 or int64, table [vocab, d] bf16, fp16 or fp32 -> the first stream
    x [..., hc_mult, d] bf16, scale * table[id] in every copy (zeros for an id outside the
    table, such as -1).  hc_mult is 1, 4 or 8."""
    dev, shape, n, size = _ids_of(ids)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise TypeError("table must be a tensor [vocab, d]")
    code = _row_type(table.dtype, "table")
    _on(table, "table", table.dtype, dev.index)
    vocab, d = table.shape
    x = _made(x, "x", shape + (int(hc_mult), d), _BF16, dev, stream)
    _run("hc_embed", dev, stream, n, int(hc_mult), d, vocab, size, code, scale, ids.data_ptr(),
         table.data_ptr(), x.data_ptr())
    return x


@functools.lru_cache(maxsize=256)
def hc_embed_backward_bytes(n: int, d: int, vocab: int) -> int:
    return int(lib().hc_embed_backward_bytes(int(n), int(d), int(vocab)))


def hc_embed_backward(dx, ids, vocab: int, scale: float = 1.0, dtable=None,
                      accumulate: bool = False, dtype=torch.float32, workspace=None, stream=None):
    """The gradient of hc_embed's table [vocab, d] from dx [..., hc, d] bf16 and ids [...].
    accumulate=False writes dtable (a new one of `dtype` where none is given) and clears the
    rows that no token names; accumulate=True adds to the given dtable.  Returns dtable."""
    dev, shape, n, size = _ids_of(ids)
    _on(dx, "dx", _BF16, dev.index)
    dims = _tokens_of(dx)
    if dims[0][:-2] != shape:
        raise ValueError("dx must be %s + (hc, d), got %s" % (shape, dims[0]))
    hc, d, vocab = dims[2], dims[3], int(vocab)
    if dtable is None and accumulate:
        raise ValueError("accumulate needs a dtable to add to")
    if dtable is not None:
        if not isinstance(dtable, torch.Tensor):
            raise TypeError("dtable must be a torch.Tensor")
        dtype = dtable.dtype
    code = _row_type(dtype, "dtable")
    dtable = _made(dtable, "dtable", (vocab, d), dtype, dev, stream)
    if workspace is None:
        workspace = _made(None, "workspace", (hc_embed_backward_bytes(n, d, vocab),), _U8, dev,
                          stream)
    else:
        _need(workspace, "workspace", _U8, dev)
    _run("hc_embed_backward", dev, stream, n, hc, d, vocab, size, code, scale, int(accumulate),
         ids.data_ptr(), dx.data_ptr(), dtable.data_ptr(), workspace.data_ptr(),
         workspace.numel())
    return dtable


def hc_launch_count() -> int:
    """Kernels the library has enqueued in this process since it was loaded."""
    return int(lib().hc_launch_count())


def hc_device_error(clear: bool = True) -> int:
    """The current device's error word (bit 0: a bounded wait timed out)."""
    v = ctypes.c_uint(0)
    _check(lib().hc_device_error(ctypes.byref(v), 1 if clear else 0), "hc_device_error")
    return int(v.value)


def hc_selftest_wait_timeout(limit_ns: int = 1000000, device=None, stream=None) -> None:
    """Enqueues the library's bounded-wait self-test: a wait that can only
    time out, after which hc_device_error() reports bit 0."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
    _check(_call(dev, lib().hc_selftest_wait_timeout, int(limit_ns), _stream(dev, stream)),
           "hc_selftest_wait_timeout")
