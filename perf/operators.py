"""The training operators of the residual-mixing path, as they are measured.

A training step keeps one residual stream [n, hc, d] per sublayer boundary,
hc times what a plain residual network keeps.  The operators keep it in 8 bits
and read it there in the backward pass:

  checkpoint       a bf16 tensor in 8 bits: e4m3 codes, one power-of-two scale
                   for each 32 channels of a row
  post_checkpoint  the expansion at the end of a sublayer, which writes the new
                   stream and its checkpoint
  restore          the bf16 tensor a checkpoint stands for
  pre_restore      the sublayer input sum_j pre_j x_j from a checkpoint: what a
                   recomputed sublayer starts from
  post_backward    gradients of the expansion
  mixes_pre_backward  gradients of the mix projection, the Sinkhorn split and
                   the collapse, with the gradient of the stream that passes
                   the sublayer by added in

`own` chooses between the plain form (elementary torch operations in 32 bits)
and the framework's kernels.
"""
import math

import torch

own = False

BLOCK = 32          # channels that share a scale
EPS, NORM_EPS = 1e-6, 1e-20
ITERS = 20


# ------------------------------------------------------------------- cases

def listed():
    def case(name, op, n, hc, d, bits=8, **more):
        return dict(name=name, op=op, n=n, hc=hc, d=d, bits=bits, **more)

    return [
        # the stream of a large training batch (8 sequences of 8,192 tokens) saved
        case("checkpoint 65536", "checkpoint", 65536, 4, 5120),
        # a short ragged batch of a narrow model: the last block of a row has 8 channels
        case("checkpoint 333 ragged", "checkpoint", 333, 4, 1000),
        # the end of a sublayer in the forward pass, one 4,096-token sequence
        case("post_checkpoint 4096", "post_checkpoint", 4096, 4, 5120),
        # eight copies, an odd count of tokens
        case("post_checkpoint 1537 hc8", "post_checkpoint", 1537, 8, 2560),
        # the whole stream back, for a sublayer recomputed with it
        case("restore 4096", "restore", 4096, 4, 5120),
        # a sublayer's input for its recomputation, straight from the checkpoint
        case("pre_restore 16384", "pre_restore", 16384, 4, 5120),
        # the backward pass at the end of a sublayer: large batch, stream and output in 8 bits
        case("post_backward 16384", "post_backward", 16384, 4, 5120, dres=False),
        # eight copies, kept in bf16, the stream's own gradient wanted as well
        case("post_backward 1001 hc8", "post_backward", 1001, 8, 1032, bits=16, dres=True),
        # the backward pass at the head of a sublayer: the large training batch
        case("mixes_pre_backward 65536", "mixes_pre_backward", 65536, 4, 5120),
        # one sequence, the stream kept in bf16
        case("mixes_pre_backward 4096 bf16", "mixes_pre_backward", 4096, 4, 5120, bits=16),
        # eight copies
        case("mixes_pre_backward 4096 hc8", "mixes_pre_backward", 4096, 8, 5120),
        # the smallest call: eight tokens of a tiny model, latency alone
        case("mixes_pre_backward 8", "mixes_pre_backward", 8, 4, 64),
    ]


def draw(rng):
    op = rng.choice(["checkpoint", "post_checkpoint", "restore", "pre_restore",
                     "post_backward", "post_backward", "mixes_pre_backward",
                     "mixes_pre_backward"])
    hc = rng.choice([4, 4, 8])
    d = 8 * int(round(math.exp(rng.uniform(math.log(8), math.log(640)))))
    most = 65536 * 4 * 5120 // (hc * d * (2 if hc == 8 else 1))
    n = int(math.exp(rng.uniform(0.0, math.log(min(65536, most)))))
    c = dict(op=op, n=max(1, n), hc=hc, d=d, bits=8)
    if op in ("post_backward", "mixes_pre_backward"):
        c["bits"] = rng.choice([8, 8, 16])
    if op == "post_backward":
        c["dres"] = rng.random() < 0.5
    return c


def work(case):
    n, hc, d, op = case["n"], case["hc"], case["d"], case["op"]
    mix = (2 + hc) * hc
    el = n * hc * d                          # stream elements
    blocks = lambda rows: rows * -(-d // BLOCK)  # noqa: E731
    kept = lambda rows: rows * d * 2 if case["bits"] == 16 else rows * d + blocks(rows)  # noqa: E731
    if op == "checkpoint":
        return {"bytes": 2 * el + el + blocks(n * hc), "flops": 2 * el}
    if op == "restore":
        return {"bytes": el + blocks(n * hc) + 2 * el, "flops": el}
    if op == "post_checkpoint":
        return {"bytes": 2 * n * d + 2 * el + 4 * n * (hc + hc * hc) + 3 * el + blocks(n * hc),
                "flops": 2 * el * (1 + hc) + 2 * el}
    if op == "pre_restore":
        return {"bytes": el + blocks(n * hc) + 4 * n * hc + 2 * n * d, "flops": 2 * el}
    if op == "post_backward":
        b = 2 * el + kept(n) + kept(n * hc) + 4 * n * (hc + hc * hc)      # read
        b += 2 * n * d + 4 * n * (hc + hc * hc) + (2 * el if case["dres"] else 0)
        return {"bytes": b, "flops": 2 * el * (2 + hc + (hc if case["dres"] else 0))}
    b = 2 * n * d + kept(n * hc) + 4 * n * mix + 4 * mix * hc * d + 4 * (3 + mix)
    b += 4 * n * (hc + hc * hc) + 2 * el                                   # read
    b += 2 * el + 4 * mix * hc * d + 4 * (3 + mix)                         # written
    return {"bytes": b, "flops": 2 * el * (2 * mix + hc + 4)}


# ------------------------------------------------------------------ inputs

def _stream(shape, g, scaled):
    """bf16 N(0, 1), each token times a scale of its own in [0.1, 10] where `scaled`."""
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for i in range(0, shape[0], 4096):
        part = t[i:i + 4096]
        v = torch.randn(part.shape, generator=g, device="cuda")
        if scaled:
            u = torch.rand((part.shape[0],) + (1,) * (len(shape) - 1), generator=g, device="cuda")
            v *= torch.exp((2 * u - 1) * math.log(10.0))
        part.copy_(v)
    return t


def _kept(t, bits):
    """What the forward pass kept of t: t itself, or its codes and scales."""
    if bits == 16:
        return t
    codes = torch.empty(t.shape, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(t.shape[:-1] + (-(-t.shape[-1] // BLOCK),), dtype=torch.uint8,
                         device="cuda")
    for i in range(0, t.shape[0], 4096):
        c, s = plain_checkpoint(t[i:i + 4096])
        codes[i:i + 4096] = c
        scales[i:i + 4096] = s
    return codes, scales


def _gradient(shape, g):
    return _stream(shape, g, False).mul_(2.0 ** -8)


def prepare(case, seed):
    n, hc, d, op, bits = case["n"], case["hc"], case["d"], case["op"], case["bits"]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    mix, F = (2 + hc) * hc, hc * d
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")    # noqa: E731
    s = {"case": dict(case)}
    x = _stream((n, hc, d), g, True)
    if op == "checkpoint":
        return s | {"x": x}
    if op == "restore":
        return s | {"kept": _kept(x, 8)}
    hc_scale, hc_base = 0.5 + 1.5 * rand(3), randn(mix)
    if op == "mixes_pre_backward":
        w = randn(mix, F) * F ** -0.5
        mixes = torch.cat([_mixes(x[i:i + 4096], w) for i in range(0, n, 4096)])
    else:
        mixes = randn(n, mix)
    pre, post, comb = plain_split(mixes, hc_scale, hc_base, hc)[:3]
    s |= {"pre": pre, "post": post, "comb": comb}
    if op == "pre_restore":
        return s | {"kept": _kept(x, 8)}
    if op == "post_checkpoint":
        return s | {"residual": x, "out": _stream((n, d), g, False)}
    s |= {"dstream": _gradient((n, hc, d), g), "residual": _kept(x, bits)}
    if op == "post_backward":
        return s | {"out": _kept(_stream((n, d), g, False), bits)}
    return s | {"dy": _gradient((n, d), g), "mixes": mixes, "w": w, "hc_scale": hc_scale,
                "hc_base": hc_base, "dpost": randn(n, hc) * 0.05,
                "dcomb": randn(n, hc, hc) * 0.05}


def _mixes(x, w):
    v = x.float().flatten(1)
    return (v @ w.t()) * torch.rsqrt(v.square().mean(1, keepdim=True) + NORM_EPS)


# -------------------------------------------------------------- plain forms

def plain_checkpoint(t):
    """codes, scales of t: the block's largest magnitude, over the scale, lies in (224, 448];
    448 is the largest e4m3 number."""
    d = t.shape[-1]
    v = torch.nn.functional.pad(t.float(), (0, -d % BLOCK)).unflatten(-1, (-1, BLOCK))
    bits = v.abs().amax(-1).view(torch.int32)
    b = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(min=1)
    v = v * ((254 - b) << 23).view(torch.float32)[..., None]
    return v.flatten(-2)[..., :d].to(torch.float8_e4m3fn).contiguous(), b.to(torch.uint8)


def plain_restore(kept):
    """The numbers that were kept, in 32 bits."""
    if isinstance(kept, torch.Tensor):
        return kept.float()
    codes, scales = kept
    f = (scales.int() << 23).view(torch.float32).repeat_interleave(BLOCK, -1)
    return codes.float() * f[..., :codes.shape[-1]]


def plain_split(mixes, hc_scale, hc_base, hc, iters=ITERS):
    """pre, post, comb; then the sigmoids, the softmax and each Sinkhorn step's (result,
    divisor)."""
    a = torch.repeat_interleave(hc_scale, torch.tensor([hc, hc, hc * hc], device=mixes.device),
                                output_size=(2 + hc) * hc)
    z = mixes * a + hc_base
    sig = torch.sigmoid(z[:, :2 * hc])
    z = z[:, 2 * hc:].unflatten(1, (hc, hc))
    e = torch.exp(z - z.amax(2, keepdim=True))
    soft = e / e.sum(2, keepdim=True)
    c, steps = soft + EPS, []
    for i in range(1, 2 * iters):
        den = c.sum(1 if i % 2 else 2, keepdim=True) + EPS
        c = c / den
        steps.append((c, den))
    return sig[:, :hc] + EPS, 2 * sig[:, hc:], c, sig, soft, steps


def plain_split_backward(dpre, dpost, dcomb, hc, sig, soft, steps):
    """The gradient of the logits, [n, (2 + hc) hc]."""
    g = dcomb
    for i in range(len(steps), 0, -1):
        c, den = steps[i - 1]
        g = (g - (g * c).sum(1 if i % 2 else 2, keepdim=True)) / den
    g = soft * (g - (g * soft).sum(2, keepdim=True))
    ds = torch.cat([dpre, 2 * dpost], 1) * sig * (1 - sig)
    return torch.cat([ds, g.flatten(1)], 1)


def plain_post(out, residual, post, comb):
    y = post[..., None] * out.float()[:, None] + comb.transpose(1, 2) @ residual.float()
    return y.to(torch.bfloat16)


def plain_post_backward(dstream, out, residual, post, comb, dres):
    g, o, r = dstream.float(), plain_restore(out), plain_restore(residual)
    got = {"dout": (post[..., None] * g).sum(1).to(torch.bfloat16),
           "dpost": (g * o[:, None]).sum(2), "dcomb": r @ g.transpose(1, 2)}
    if dres:
        got["dresidual"] = (comb @ g).to(torch.bfloat16)
    return got


def plain_mixes_pre_backward(dy, x, mixes, w, hc_scale, hc_base, dpost, dcomb, dstream):
    x, dy = plain_restore(x), dy.float()
    n, hc, d = x.shape
    F = hc * d
    r2 = 1.0 / (x.flatten(1).square().mean(1, keepdim=True) + NORM_EPS)
    pre, _, comb, sig, soft, steps = plain_split(mixes, hc_scale, hc_base, hc)
    dpre = (x @ dy[..., None]).squeeze(2)
    dz = plain_split_backward(dpre, dpost, dcomb, hc, sig, soft, steps)
    part = [hc, hc, hc * hc]
    dscale = torch.stack([v.sum() for v in (dz * mixes).split(part, 1)])
    dm = torch.cat([v * hc_scale[i] for i, v in enumerate(dz.split(part, 1))], 1)
    du = dm * torch.sqrt(r2)
    q = -(dm * mixes).sum(1, keepdim=True) * r2 / F
    dx = pre[..., None] * dy[:, None] + q[..., None] * x
    dx += (du @ w).view(n, hc, d)
    dx += comb @ dstream.float()
    return {"dx": dx.to(torch.bfloat16), "dw": du.t() @ x.flatten(1), "dscale": dscale,
            "dbase": dz.sum(0)}


# --------------------------------------------------------------------- run

def run(s):
    c = s["case"]
    op, hc = c["op"], c["hc"]
    if own:
        import sinkhorn_mixing_gb300 as lib
        if op == "checkpoint":
            codes, scales = lib.hc_checkpoint(s["x"])
            return {"codes": codes, "scales": scales}
        if op == "restore":
            return {"x": lib.hc_restore(*s["kept"])}
        if op == "pre_restore":
            return {"y": lib.hc_pre_restore(*s["kept"], s["pre"])}
        if op == "post_checkpoint":
            y, codes, scales = lib.hc_post_checkpoint(s["out"], s["residual"], s["post"],
                                                      s["comb"])
            return {"y": y, "codes": codes, "scales": scales}
        if op == "post_backward":
            got = lib.hc_post_backward(s["dstream"], s["out"], s["residual"], s["post"],
                                       s["comb"], want_dresidual=c["dres"])
            return dict(zip(("dout", "dpost", "dcomb", "dresidual"), got[:4 if c["dres"] else 3]))
        got = lib.hc_mixes_pre_backward(s["dy"], s["residual"], s["mixes"], s["w"],
                                        s["hc_scale"], s["hc_base"], s["dpost"], s["dcomb"],
                                        dstream=s["dstream"], sinkhorn_iters=ITERS, eps=EPS,
                                        norm_eps=NORM_EPS)
        return dict(zip(("dx", "dw", "dscale", "dbase"), got))
    if op == "checkpoint":
        codes, scales = plain_checkpoint(s["x"])
        return {"codes": codes, "scales": scales}
    if op == "restore":
        return {"x": plain_restore(s["kept"]).to(torch.bfloat16)}
    if op == "pre_restore":
        return {"y": (s["pre"][:, None] @ plain_restore(s["kept"])).squeeze(1).to(torch.bfloat16)}
    if op == "post_checkpoint":
        y = plain_post(s["out"], s["residual"], s["post"], s["comb"])
        codes, scales = plain_checkpoint(y)
        return {"y": y, "codes": codes, "scales": scales}
    if op == "post_backward":
        return plain_post_backward(s["dstream"], s["out"], s["residual"], s["post"], s["comb"],
                                   c["dres"])
    return plain_mixes_pre_backward(s["dy"], s["residual"], s["mixes"], s["w"], s["hc_scale"],
                                    s["hc_base"], s["dpost"], s["dcomb"], s["dstream"])


# ------------------------------------------------------- 64-bit definitions

def _kept64(kept):
    if isinstance(kept, torch.Tensor):
        return kept.double()
    codes, scales = kept
    of = torch.arange(codes.shape[-1], device="cuda") // BLOCK
    return codes.float().double() * torch.exp2(scales.double() - 127.0)[..., of]


def _cut(kept, i, j):
    return kept[i:j] if isinstance(kept, torch.Tensor) else tuple(k[i:j] for k in kept)


def _comb64(z, iters):
    """comb of the logits z [n, hc, hc], from its definition."""
    c = torch.softmax(z, 2) + EPS
    c = c / (c.sum(1, keepdim=True) + EPS)
    for _ in range(iters - 1):
        c = c / (c.sum(2, keepdim=True) + EPS)
        c = c / (c.sum(1, keepdim=True) + EPS)
    return c


def exact(case, seed):
    """From the definitions in 64 bits; gradients by automatic differentiation of them."""
    s = prepare(case, seed)
    op, n, hc, d = case["op"], case["n"], case["hc"], case["d"]
    step = max(1, (1 << 26) // (hc * d))
    cuts = [(i, min(n, i + step)) for i in range(0, n, step)]
    if op == "checkpoint":
        # no rounding: the block's numbers over its scale, the smallest power of two that
        # brings all of them to 448 or less
        got = []
        for i, j in cuts:
            v = torch.nn.functional.pad(s["x"][i:j].double(), (0, -d % BLOCK)).unflatten(
                -1, (-1, BLOCK))
            e = torch.ceil(torch.log2(v.abs().amax(-1, keepdim=True) / 448.0)).clamp(min=-126)
            got.append((v * torch.exp2(-e)).flatten(-2)[..., :d])
        return {"codes": torch.cat(got), "scales": None}
    if op == "restore":
        return {"x": torch.cat([_kept64(_cut(s["kept"], i, j)) for i, j in cuts])}
    if op == "pre_restore":
        return {"y": torch.cat([torch.einsum("nj,njc->nc", s["pre"][i:j].double(),
                                             _kept64(_cut(s["kept"], i, j))) for i, j in cuts])}
    post, comb = s["post"].double(), s["comb"].double()
    if op == "post_checkpoint":
        y = [torch.einsum("nk,nc->nkc", post[i:j], s["out"][i:j].double()) +
             torch.einsum("njk,njc->nkc", comb[i:j], s["residual"][i:j].double())
             for i, j in cuts]
        return {"y": torch.cat(y), "codes": None, "scales": None}
    if op == "post_backward":
        parts = {"dout": [], "dpost": [], "dcomb": []} | ({"dresidual": []} if case["dres"] else {})
        for i, j in cuts:
            o = _kept64(_cut(s["out"], i, j)).requires_grad_()
            r = _kept64(_cut(s["residual"], i, j)).requires_grad_()
            p, c = (t[i:j].clone().requires_grad_() for t in (post, comb))
            y = p[..., None] * o[:, None] + torch.einsum("njk,njc->nkc", c, r)
            grads = torch.autograd.grad(y, (o, p, c, r), s["dstream"][i:j].double())
            for key, t in zip(("dout", "dpost", "dcomb", "dresidual"), grads):
                if key in parts:
                    parts[key].append(t)
        return {k: torch.cat(v) for k, v in parts.items()}
    F = hc * d
    w = s["w"].double()
    scale, base = (s[k].double().requires_grad_() for k in ("hc_scale", "hc_base"))
    dw, dscale, dbase, dx = torch.zeros_like(w), 0.0, 0.0, []
    for i, j in cuts:
        x = _kept64(_cut(s["residual"], i, j)).requires_grad_()
        v = x.flatten(1)
        r = (v.square().mean(1, keepdim=True) + NORM_EPS) ** -0.5
        # the projection's value is the mix numbers the forward pass kept; its derivatives are
        # those at the stream that was kept
        u = (s["mixes"][i:j].double() / r).detach().requires_grad_()
        m = r * u
        z = torch.cat([m[:, :hc] * scale[0], m[:, hc:2 * hc] * scale[1], m[:, 2 * hc:] * scale[2]],
                      1) + base
        pre = torch.sigmoid(z[:, :hc]) + EPS
        po = 2 * torch.sigmoid(z[:, hc:2 * hc])
        co = _comb64(z[:, 2 * hc:].unflatten(1, (hc, hc)), ITERS)
        y = torch.einsum("nj,njc->nc", pre, x)
        past = torch.einsum("njk,njc->nkc", co.detach(), x)
        grads = torch.autograd.grad(
            (y, past, po, co), (x, u, scale, base),
            (s["dy"][i:j].double(), s["dstream"][i:j].double(), s["dpost"][i:j].double(),
             s["dcomb"][i:j].double()))
        du = grads[1]
        dx.append(grads[0] + (du @ w).view(j - i, hc, d))
        dw += du.t() @ v.detach()
        dscale, dbase = dscale + grads[2], dbase + grads[3]
    return {"dx": torch.cat(dx), "dw": dw, "dscale": dscale, "dbase": dbase}
