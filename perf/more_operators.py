"""The operators at the two ends of a sublayer's training step, as they are measured.

A training step of the residual-mixing path starts with the tokens' rows of the
embedding table, put into every copy of the stream, and each sublayer reads its input
through a norm.  The operators are those two, with their gradients:

  norm            y = (x - mean) / sqrt(variance + eps) * weight + bias over each row
                  (layer norm), or without the mean (RMS norm, the framework's)
  norm_backward   gradients of the rows, the weight and the bias; the last two are sums
                  over all rows
  embed           scale * table[id] for each token, in bf16, written to all copies of its
                  stream; an id outside the table (padding, -1) gives zeros
  embed_backward  the table's gradient: the stream's gradient summed over the copies and
                  over the tokens that share an id.  With two micro-batches the first is
                  written (rows that no token names become zero) and the second added

`own` chooses between the plain form (elementary torch operations in 32 bits) and the
framework's kernels.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = {False: 1e-20, True: 1e-5}    # the RMS norm's as the framework has it; layer norm's usual one


# ------------------------------------------------------------------- cases

def listed():
    def norm(name, op, rows, d, type="bf16", center=False, bias=False):
        return dict(name=name, op=op, rows=rows, d=d, type=type, center=center, bias=bias)

    def embed(name, op, n, hc, d, vocab, type="bf16", scaled=False, pad=False, ids=64, parts=1):
        return dict(name=name, op=op, n=n, hc=hc, d=d, vocab=vocab, type=type, scaled=scaled,
                    pad=pad, ids=ids, parts=parts)

    return [
        # the sublayer input of a large training batch (8 sequences of 8,192 tokens)
        norm("norm 65536", "norm", 65536, 5120),
        # a decode step of 64 requests: latency alone
        norm("norm 64", "norm", 64, 5120),
        # a norm per attention head: many short rows
        norm("norm 131072 x 128", "norm", 131072, 128),
        # layer norm with a bias in fp16, an odd count of rows of a narrow model
        norm("norm 1001 ragged layer", "norm", 1001, 1000, "fp16", True, True),
        # the large training batch's backward pass
        norm("norm_backward 65536", "norm_backward", 65536, 5120),
        # one sequence, layer norm with a bias
        norm("norm_backward 4096 layer", "norm_backward", 4096, 5120, "bf16", True, True),
        # a short ragged batch kept in fp32
        norm("norm_backward 333 fp32 layer", "norm_backward", 333, 1000, "fp32", True, True),
        # the first stream of a large training batch
        embed("embed 65536", "embed", 65536, 4, 5120, 131072),
        # a decode step of 64 requests from a table kept in fp32, scaled, with idle slots
        embed("embed 64 fp32", "embed", 64, 4, 5120, 32768, "fp32", True, True, ids=32),
        # the table's gradient at the end of a large training batch, kept in fp32
        embed("embed_backward 65536", "embed_backward", 65536, 4, 5120, 131072, "fp32"),
        # two micro-batches of one sequence each into a gradient in bf16
        embed("embed_backward 2 x 4096", "embed_backward", 4096, 4, 5120, 32768, "bf16", parts=2),
        # eight copies, odd sizes, padding among the tokens
        embed("embed_backward 1537 hc8", "embed_backward", 1537, 8, 1032, 50001, "fp32", True, True),
    ]


def draw(rng):
    def over(low, high):
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    op = rng.choice(["norm", "norm_backward", "embed", "embed_backward"])
    if op.startswith("norm"):
        d = 8 * over(1, 2560)
        center = rng.random() < 0.5
        kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = 65536 * 5120 * 2 // (d * SIZE[kind])
        return dict(op=op, rows=over(1, min(262144, most)), d=d, type=kind, center=center,
                    bias=center and rng.random() < 0.75)
    hc = rng.choice([1, 4, 4, 8])
    d = 8 * over(8, 640)
    kind = rng.choice(["bf16", "fp16", "fp32"])
    parts = 2 if op == "embed_backward" and rng.random() < 0.3 else 1
    n = over(1, min(65536, 65536 * 4 * 5120 // (hc * d * parts)))
    vocab = over(100, min(131072, 131072 * 5120 // d))
    return dict(op=op, n=n, hc=hc, d=d, vocab=vocab, type=kind, scaled=rng.random() < 0.5,
                pad=rng.random() < 0.5, ids=rng.choice([32, 64]), parts=parts)


def _named(vocab, n, pad):
    """How many distinct ids n drawn tokens are expected to name (see _ids)."""
    v = np.arange(vocab, dtype=np.float64)
    p = np.log1p(1.0 / (v + 1.0)) / math.log(vocab + 1.0) * (1.0 - (1.0 / 16 if pad else 0.0))
    return float(-np.expm1(n * np.log1p(-p)).sum()) if vocab > 1 else 1.0


def work(case):
    op, d, size = case["op"], case["d"], SIZE[case["type"]]
    if op.startswith("norm"):
        el = case["rows"] * d
        par = 4 * d * (2 if case["bias"] else 1)
        if op == "norm":
            return {"bytes": 2 * size * el + par, "flops": el * (7 if case["center"] else 4)}
        return {"bytes": 3 * size * el + 4 * d + par, "flops": el * (14 if case["center"] else 9)}
    n, hc, vocab, parts = case["n"], case["hc"], case["vocab"], case["parts"]
    el = n * hc * d
    ids = n * case["ids"] // 8
    named = _named(vocab, n, case["pad"]) * d * size
    if op == "embed":
        return {"bytes": 2 * el + named + ids, "flops": n * d}
    # each micro-batch's gradients read; the first writes the table, the others read and write
    # the rows they name
    return {"bytes": parts * (2 * el + ids) + vocab * d * size + (parts - 1) * 2 * named,
            "flops": parts * el + vocab * d}


# ------------------------------------------------------------------ inputs

def _normal(shape, type, g, scale=1.0, spread=False):
    """N(0, scale^2), each row times a factor of its own in [0.1, 10] where `spread`."""
    t = torch.empty(shape, dtype=type, device="cuda")
    step = max(1, (1 << 26) // (t[0].numel() if shape[0] else 1))
    for i in range(0, shape[0], step):
        v = torch.randn((min(step, shape[0] - i),) + tuple(shape[1:]), generator=g, device="cuda")
        if spread:
            u = torch.rand((v.shape[0],) + (1,) * (v.dim() - 1), generator=g, device="cuda")
            v *= torch.exp((2 * u - 1) * math.log(10.0))
        t[i:i + step] = v.mul_(scale)
    return t


def _ids(n, vocab, pad, bits, g):
    """Tokens as texts have them: id v with probability ln((v + 2) / (v + 1)) / ln(vocab + 1), a
    few ids in most places and a long tail; one in sixteen is padding (-1) where `pad`."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(vocab + 1.0)).floor().long() - 1).clamp(0, vocab - 1)
    if pad:
        ids[torch.rand(n, generator=g, device="cuda") < 1.0 / 16] = -1
    return ids.to(torch.int32 if bits == 32 else torch.int64)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    op, d, type = case["op"], case["d"], TYPES[case["type"]]
    s = {"case": dict(case)}
    if op.startswith("norm"):
        rows = case["rows"]
        s["x"] = _normal((rows, d), type, g, spread=True)
        if case["center"]:
            s["x"] += torch.randn(rows, 1, generator=g, device="cuda").to(type)
        s["weight"] = 0.5 + torch.rand(d, generator=g, device="cuda")
        s["bias"] = torch.randn(d, generator=g, device="cuda") if case["bias"] else None
        if op == "norm_backward":
            s["dy"] = _normal((rows, d), type, g, 2.0 ** -8)
        return s
    n, hc, vocab, parts = case["n"], case["hc"], case["vocab"], case["parts"]
    s["scale"] = float(np.float32(math.sqrt(d))) if case["scaled"] else 1.0
    s["ids"] = [_ids(n, vocab, case["pad"], case["ids"], g) for _ in range(parts)]
    if op == "embed":
        s["table"] = _normal((vocab, d), type, g, 1.0 / s["scale"])
    else:
        s["dx"] = [_normal((n, hc, d), torch.bfloat16, g, 2.0 ** -8) for _ in range(parts)]
    return s


# -------------------------------------------------------------- plain forms

def _centered(x, center, eps):
    """The row without its mean, and one over its standard deviation, in 32 bits."""
    v = x.float()
    if center:
        v = v - v.mean(1, keepdim=True)
    return v, torch.rsqrt(v.square().mean(1, keepdim=True) + eps)


def plain_norm(x, weight, bias, center, eps):
    v, r = _centered(x, center, eps)
    y = v * r * weight
    if bias is not None:
        y = y + bias
    return y.to(x.dtype)


def plain_norm_backward(dy, x, weight, center, bias, eps):
    v, r = _centered(x, center, eps)
    h, dy = v * r, dy.float()
    g = dy * weight
    dx = g - h * (g * h).mean(1, keepdim=True)
    if center:
        dx = dx - g.mean(1, keepdim=True)
    out = {"dx": (dx * r).to(x.dtype), "dweight": (dy * h).sum(0)}
    if bias:
        out["dbias"] = dy.sum(0)
    return out


def plain_embed(ids, table, hc, scale):
    inside = (ids >= 0) & (ids < table.shape[0])
    x = table[ids.long().clamp(0, table.shape[0] - 1)].float() * scale
    x = torch.where(inside[:, None], x, torch.zeros((), device=x.device)).to(torch.bfloat16)
    return x[:, None].repeat(1, hc, 1)


def plain_embed_backward(parts, vocab, d, type, scale):
    table = None
    for ids, dx in parts:
        inside = ((ids >= 0) & (ids < vocab)).nonzero().squeeze(1)
        rows = dx.sum(1, dtype=torch.float32)[inside]
        got = torch.zeros(vocab, d, device=dx.device).index_add_(0, ids.long()[inside], rows)
        got *= scale
        table = (got if table is None else table.float() + got).to(type)
    return table


# --------------------------------------------------------------------- run

def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import sinkhorn_mixing_gb300 as lib
        if op == "norm":
            return {"y": lib.hc_norm(s["x"], s["weight"], s["bias"], eps=EPS[c["center"]],
                                     center=c["center"])}
        if op == "norm_backward":
            got = lib.hc_norm_backward(s["dy"], s["x"], s["weight"], eps=EPS[c["center"]],
                                       center=c["center"], want_dbias=c["bias"])
            return dict(zip(("dx", "dweight", "dbias"), got[:3 if c["bias"] else 2]))
        if op == "embed":
            return {"x": lib.hc_embed(s["ids"][0], s["table"], hc_mult=c["hc"], scale=s["scale"])}
        dtable = None
        for ids, dx in zip(s["ids"], s["dx"]):
            dtable = lib.hc_embed_backward(dx, ids, c["vocab"], scale=s["scale"], dtable=dtable,
                                           accumulate=dtable is not None, dtype=TYPES[c["type"]])
        return {"dtable": dtable}
    if op == "norm":
        return {"y": plain_norm(s["x"], s["weight"], s["bias"], c["center"], EPS[c["center"]])}
    if op == "norm_backward":
        return plain_norm_backward(s["dy"], s["x"], s["weight"], c["center"], c["bias"],
                                   EPS[c["center"]])
    if op == "embed":
        return {"x": plain_embed(s["ids"][0], s["table"], c["hc"], s["scale"])}
    return {"dtable": plain_embed_backward(list(zip(s["ids"], s["dx"])), c["vocab"], c["d"],
                                           TYPES[c["type"]], s["scale"])}


# ------------------------------------------------------- 64-bit definitions

def _norm64(x, weight, bias, center, eps):
    m = x.mean(1, keepdim=True) if center else 0.0
    y = (x - m) / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + eps) * weight
    return y if bias is None else y + bias


def exact(case, seed):
    """From the definitions in 64 bits; gradients by automatic differentiation of them."""
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op.startswith("norm"):
        center = case["center"]
        w = s["weight"].double().requires_grad_()
        b = torch.zeros_like(w) if s["bias"] is None else s["bias"].double()
        b = b.detach().requires_grad_()
        step = max(1, (1 << 26) // d)
        out, dw, db = [], 0.0, 0.0
        for i in range(0, case["rows"], step):
            x = s["x"][i:i + step].double().requires_grad_(op == "norm_backward")
            if op == "norm":
                with torch.no_grad():
                    out.append(_norm64(x, w, b, center, EPS[center]))
                continue
            y = _norm64(x, w, b, center, EPS[center])
            gx, gw, gb = torch.autograd.grad(y, (x, w, b), s["dy"][i:i + step].double())
            out.append(gx)
            dw, db = dw + gw, db + gb
        if op == "norm":
            return {"y": torch.cat(out)}
        return {"dx": torch.cat(out), "dweight": dw} | ({"dbias": db} if case["bias"] else {})
    n, hc, vocab = case["n"], case["hc"], case["vocab"]
    if op == "embed":
        ids = s["ids"][0].long()
        # a row of zeros behind the table for the tokens that name none
        full = torch.cat([s["table"], s["table"].new_zeros(1, d)])
        rows = full[torch.where((ids < 0) | (ids >= vocab), vocab, ids)].double() * s["scale"]
        return {"x": rows[:, None].expand(n, hc, d)}
    out = torch.zeros(vocab, d, dtype=torch.float64, device="cuda")
    for ids, dx in zip(s["ids"], s["dx"]):
        ids = ids.long()
        ids = torch.where((ids < 0) | (ids >= vocab), vocab, ids)
        order = torch.argsort(ids, stable=True)
        count = torch.bincount(ids, minlength=vocab + 1)[:vocab]
        at = torch.cumsum(count, 0)
        for j in range(0, d, 512):
            # the sum over an id's tokens: a difference of running sums over the sorted tokens
            run = torch.cumsum(dx[..., j:j + 512].double().sum(1)[order], 0)
            run = torch.cat([run.new_zeros(1, run.shape[1]), run])
            out[:, j:j + 512] += (run[at] - run[at - count]) * s["scale"]
    return {"dtable": out}
