"""Workloads around the FP8 Linear in a training step: the embedding at its start, the softmax cross entropy of the
head's product at its end, and the norm and SwiGLU between, whose backward passes read activations kept in 8 bits; each
in a plain form of elementary torch operations and through the library."""
import math

import torch

own = False

_FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
_FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _xent(name, part, tokens, vocab, dim, ignored=0.0, scale=1.0, zloss=0):
    return {"name": name, "op": "xent", "part": part, "tokens": tokens, "vocab": vocab, "dim": dim, "ignored": ignored,
            "scale": scale, "zloss": zloss}


def _embed(name, part, tokens, vocab, dim, grad="f32", accumulate=1, scale=1.0):
    return {"name": name, "op": "embed", "part": part, "tokens": tokens, "vocab": vocab, "dim": dim, "grad": grad,
            "accumulate": accumulate, "scale": scale}


def _norm(name, part, rows, cols, fmt="e4m3", residual=1):
    return {"name": name, "op": "norm", "part": part, "rows": rows, "cols": cols, "fmt": fmt, "residual": residual}


def _swiglu(name, part, rows, ffn, fmt="e4m3"):
    return {"name": name, "op": "swiglu", "part": part, "rows": rows, "ffn": ffn, "fmt": fmt}


def listed():
    return [
        # scoring a handful of tokens with a small head: the call's latency
        _xent("xent_score_4", "fwd", 4, 8000, 1024),
        # scoring one token of each request of a batch: the head's weights are read once
        _xent("xent_score_64", "fwd", 64, 128000, 4096),
        # a fine-tuning batch: half the tokens are prompt and do not count, a tempered head
        _xent("xent_masked_4000", "fwd", 4000, 32001, 2048, ignored=0.5, scale=0.7),
        # gradient of a short ragged batch
        _xent("xent_grad_300", "bwd", 300, 50001, 1536),
        # a whole training step's loss and gradients at the benchmark's 8192 tokens and hidden size
        _xent("xent_step_8192", "both", 8192, 128000, 4096, zloss=1),
        # the step's tokens looked up
        _embed("embed_8192", "fwd", 8192, 128000, 4096, scale=64.0),
        # gradient of a small batch, added to the one of the tied head
        _embed("embed_grad_1000", "bwd", 1000, 32001, 1024),
        # gradient of a large batch, the whole table written for the optimizer
        _embed("embed_grad_32768", "bwd", 32768, 128000, 2048, grad="bf16", accumulate=0),
        # residual added and normalised, the sum kept in 8 bits, at the benchmark's sizes
        _norm("norm_fwd_8192", "fwd", 8192, 4096),
        # its backward pass from the 8-bit sum
        _norm("norm_bwd_8192", "bwd", 8192, 4096),
        # a few rows of a small model: the call's latency
        _swiglu("swiglu_fwd_40", "fwd", 40, 1408),
        # backward of the benchmark's MLP activation from its 8-bit checkpoint
        _swiglu("swiglu_bwd_8192", "bwd", 8192, 14336),
    ]


def _spread(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["xent", "xent", "embed", "norm", "swiglu"])
    part = rng.choice(["fwd", "bwd"])
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    if op == "xent":
        part = rng.choice(["fwd", "bwd", "both"])
        dim, vocab = _spread(rng, 128, 4096, 8), _spread(rng, 1000, 128000)
        most = int(8192 * 128000 * 4096 / 4 / (dim * vocab))
        c = _xent("", part, _spread(rng, 1, max(1, min(8192, most))), vocab, dim, rng.choice([0.0, 0.0, 0.1, 0.6]),
                  rng.choice([1.0, 1.0, 0.25]), rng.randrange(2))
    elif op == "embed":
        dim = _spread(rng, 64, 4096, 8)
        grad = rng.choice(["f32", "bf16"])
        c = _embed("", part, _spread(rng, 1, 32768), _spread(rng, 1000, 128000), dim, grad,
                   rng.randrange(2) if grad == "f32" else 0, rng.choice([1.0, 64.0]))
    elif op == "norm":
        c = _norm("", part, _spread(rng, 1, 8192), _spread(rng, 256, 8192, 128), fmt, rng.randrange(2))
    else:
        c = _swiglu("", part, _spread(rng, 1, 8192), _spread(rng, 128, 14336, 128), fmt)
    del c["name"]
    return c


def _skipped(case):
    """Tokens of a cross entropy that do not count."""
    return min(case["tokens"] - 1, int(case["tokens"] * case["ignored"]))


def work(case):
    op, part = case["op"], case["part"]
    if op == "xent":
        n, V, D = case["tokens"] - _skipped(case), case["vocab"], case["dim"]
        b, f = n * D * 2 + V * D * 2 + case["tokens"] * 12, 0
        if part != "bwd":
            f += 2 * n * V * D
        if part != "fwd":       # the logits once more, the two products of their gradient, dx and dw
            f += 6 * n * V * D
            b += case["tokens"] * D * 2 + V * D * 2
        return {"bytes": b, "flops": f}
    if op == "embed":
        T, V, D = case["tokens"], case["vocab"], case["dim"]
        if part == "fwd":
            return {"bytes": T * (4 + 4 * D), "flops": T * D}
        if case["accumulate"]:  # every row that occurs is read and written; their number goes by the seed, about:
            rows = min(V, T) * 0.4
            return {"bytes": T * (4 + 2 * D) + rows * D * 8, "flops": 2 * T * D}
        return {"bytes": T * (4 + 2 * D) + V * D * (4 if case["grad"] == "f32" else 2), "flops": 2 * T * D}
    if op == "norm":
        n, C = case["rows"] * case["cols"], case["cols"]
        if part == "fwd":
            return {"bytes": n * (4 + 1 + (4 if case["residual"] else 0)) + n // 32 + case["rows"] * 4 + C * 2, "flops": 8 * n}
        return {"bytes": n * (1 + 4 + (2 if case["residual"] else 0)) + n // 32 + case["rows"] * 4 + C * 6, "flops": 12 * n}
    n = case["rows"] * case["ffn"]
    return {"bytes": n * (4 + 2 + 2) + n // 16, "flops": n * 10} if part == "fwd" else {"bytes": n * (2 + 2 + 4) + n // 16, "flops": n * 20}


class _State:
    pass


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, by=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(by)

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, device="cuda", dtype=dtype)

    s = _State()
    s.case = case
    op, part, f32 = case["op"], case["part"], torch.float32
    if op == "xent":
        T, V, D = case["tokens"], case["vocab"], case["dim"]
        s.w = normal(V, D, by=1.5 * D ** -0.5)
        target = torch.randint(V, (T,), generator=g, device="cuda")
        # tokens from badly to well predicted: up to 16 on the target's logit
        lift = torch.rand((T, 1), generator=g, device="cuda") * (16 / 2.25)
        s.x = (torch.randn((T, D), generator=g, device="cuda") + lift * s.w[target].float()).bfloat16()
        target[torch.randperm(T, generator=g, device="cuda")[:_skipped(case)]] = -100
        s.target = target.to(torch.int32)
        s.loss, s.lse = empty(T, dtype=f32), empty(T, dtype=f32)
        if part != "fwd":
            s.dloss = (torch.rand(T, generator=g, device="cuda") + 0.5) / T
            s.dlse = torch.rand(T, generator=g, device="cuda") * (0.01 / T) if case["zloss"] else None
            s.dx, s.dw = empty(T, D), empty(V, D)
            if part == "bwd":   # the forward pass has left them
                s.loss, s.lse = _xent_forward(s)[:2]
    elif op == "embed":
        T, V, D = case["tokens"], case["vocab"], case["dim"]
        # few words make up most of a text; a row in a hundred is padding
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        word = torch.randperm(V, generator=g, device="cuda")
        ids = word[(V ** u).long().clamp_(max=V) - 1].to(torch.int32)
        s.ids = torch.where(torch.rand(T, generator=g, device="cuda") < 0.01, -1, ids)
        if part == "fwd":
            s.w, s.out = normal(V, D, by=D ** -0.5), empty(T, D)
        else:
            s.dout = normal(T, D, by=1e-3)
            s.dw = empty(V, D, dtype=f32 if case["grad"] == "f32" else torch.bfloat16)
            if case["accumulate"]:
                s.dw.normal_(generator=g).mul_(1e-3)
    elif op == "norm":
        R, C, kind = case["rows"], case["cols"], _FP8[case["fmt"]]
        s.eps = 1e-5
        s.w = (1 + 0.1 * torch.randn(C, generator=g, device="cuda")).bfloat16()
        x, res = normal(R, C), normal(R, C, by=2.0)
        res[:, ::97] *= 20.0    # the few large channels of a residual stream
        s.c, s.cs, s.rstd = empty(R, C, dtype=kind), empty(C // 128, R, dtype=f32), empty(R, dtype=f32)
        if part == "fwd":
            s.x, s.res = (x, res) if case["residual"] else (res, None)
            s.y, s.sum = empty(R, C), empty(R, C) if case["residual"] else None
        else:
            h = (x.float() + res.float()).bfloat16()
            s.rstd = torch.rsqrt(h.float().square().mean(1) + s.eps)
            s.c, s.cs = _kept(h, case["fmt"])
            s.dy, s.dsum = normal(R, C, by=1e-2), normal(R, C, by=1e-2) if case["residual"] else None
            s.dx, s.dw = empty(R, C), empty(C, dtype=f32)
    else:
        R, F, kind = case["rows"], case["ffn"], _FP8[case["fmt"]]
        gu = normal(R, 2 * F, by=1.5)
        if part == "fwd":
            s.gu, s.h = gu, empty(R, F)
            s.c, s.cs = empty(R, 2 * F, dtype=kind), empty(2 * F // 128, R, dtype=f32)
        else:
            s.c, s.cs = _kept(gu, case["fmt"])
            s.dh, s.dgu = normal(R, F, by=1e-2), empty(R, 2 * F)
    if own:
        import fp8_fine_grained_x128_gb300 as fg
        if op == "xent":
            s.workspace = fg.new_linear_xent_workspace(T, V, D, backward=part != "fwd")
        elif op == "embed" and part == "bwd":
            s.workspace = fg.new_embedding_workspace(T, V, D)
        elif op == "norm" and part == "bwd":
            s.workspace = fg.new_rmsnorm_workspace(C)
        if op in ("norm", "swiglu"):
            s.fmt = fg.E4M3 if case["fmt"] == "e4m3" else fg.E5M2
    return s


# ---------------------------------------------------------------- plain forms

def _xent_forward(s):
    logits = s.x.float() @ s.w.float().T
    logits *= s.case["scale"]
    counts = s.target >= 0
    at = s.target.clamp(min=0).long()[:, None]
    top = logits.amax(1, keepdim=True)
    lse = (logits - top).exp_().sum(1, keepdim=True).log_() + top
    loss = lse - logits.gather(1, at)
    return torch.where(counts, loss[:, 0], 0.0), torch.where(counts, lse[:, 0], 0.0), logits


def _xent_backward(s, lse, logits):
    counts = (s.target >= 0)[:, None]
    dloss = torch.where(counts, s.dloss[:, None], 0.0)
    both = dloss if s.dlse is None else dloss + torch.where(counts, s.dlse[:, None], 0.0)
    p = logits.sub_(lse[:, None]).exp_().mul_(both * s.case["scale"])
    p.scatter_add_(1, s.target.clamp(min=0).long()[:, None], dloss * -s.case["scale"])
    p.masked_fill_(~counts, 0.0)
    return (p @ s.w.float()).bfloat16(), (p.T @ s.x.float()).bfloat16()


def _xent_plain(s):
    part = s.case["part"]
    loss, lse, logits = _xent_forward(s)
    if part == "fwd":
        return loss, lse
    dx, dw = _xent_backward(s, lse if part == "both" else s.lse, logits)
    return (dx, dw) if part == "bwd" else (loss, lse, dx, dw)


def _embed_plain(s):
    case = s.case
    here = (s.ids >= 0)[:, None]
    at = s.ids.clamp(min=0).long()
    if case["part"] == "fwd":
        return torch.where(here, s.w[at].float() * case["scale"], 0.0).bfloat16()
    rows = torch.where(here, s.dout.float(), 0.0)
    dw = torch.zeros((case["vocab"], case["dim"]), device="cuda").index_add_(0, at, rows).mul_(case["scale"])
    s.dw.copy_(s.dw + dw if case["accumulate"] else dw)
    return s.dw


def _kept(x, fmt):
    """Codes and scales [columns / 128, rows] of a tensor kept in 8 bits."""
    t = x.float().unflatten(1, (-1, 128))
    amax = t.abs().amax(2)
    s = torch.where(amax == 0, 1.0, amax / _FMAX[fmt])
    return (t / s[..., None]).flatten(1).to(_FP8[fmt]), s.T.contiguous()


def _values(c, cs):
    return (c.float().unflatten(1, (-1, 128)) * cs.T[..., None]).flatten(1)


def _norm_plain(s):
    case, w = s.case, s.w.float()
    if case["part"] == "fwd":
        h = s.x if s.res is None else (s.x.float() + s.res.float()).bfloat16()
        c, cs = _kept(h, case["fmt"])
        x = h.float()
        rstd = torch.rsqrt(x.square().mean(1) + s.eps)
        y = (x * rstd[:, None] * w).bfloat16()
        return (y, c, cs, rstd) if s.res is None else (y, c, cs, rstd, h)
    x = _values(s.c, s.cs) * s.rstd[:, None]
    dy = s.dy.float()
    dn = dy * w
    dx = (dn - x * (dn * x).mean(1, keepdim=True)) * s.rstd[:, None]
    if s.dsum is not None:
        dx += s.dsum.float()
    return dx.bfloat16(), (dy * x).sum(0)


def _swiglu_plain(s):
    if s.case["part"] == "fwd":
        g, u = s.gu.float().chunk(2, 1)
        return ((g / (1 + torch.exp(-g)) * u).bfloat16(), *_kept(s.gu, s.case["fmt"]))
    g, u = _values(s.c, s.cs).chunk(2, 1)
    sig, d = 1 / (1 + torch.exp(-g)), s.dh.float()
    return torch.cat([d * u * sig * (1 + g * (1 - sig)), d * g * sig], 1).bfloat16()


_PLAIN = {"xent": _xent_plain, "embed": _embed_plain, "norm": _norm_plain, "swiglu": _swiglu_plain}


def run(state):
    s, case = state, state.case
    op, part = case["op"], case["part"]
    if not own:
        return _PLAIN[op](s)
    import fp8_fine_grained_x128_gb300 as fg
    if op == "xent":
        if part != "bwd":
            fg.linear_xent_fwd(s.x, s.w, s.target, s.loss, s.lse, s.workspace, scale=case["scale"])
        if part == "fwd":
            return s.loss, s.lse
        fg.linear_xent_bwd(s.x, s.w, s.target, s.loss, s.lse, s.dloss, s.dx, s.dw, s.workspace, dlse=s.dlse, scale=case["scale"])
        return (s.dx, s.dw) if part == "bwd" else (s.loss, s.lse, s.dx, s.dw)
    if op == "embed":
        if part == "fwd":
            fg.embedding_fwd(s.ids, s.w, s.out, scale=case["scale"])
            return s.out
        fg.embedding_bwd(s.ids, s.dout, s.dw, s.workspace, scale=case["scale"], accumulate=bool(case["accumulate"]))
        return s.dw
    if op == "norm":
        if part == "fwd":
            fg.rmsnorm_fwd_ckpt(s.x, s.w, s.eps, s.fmt, s.y, s.c, s.cs, s.rstd, res=s.res, sum=s.sum)
            return (s.y, s.c, s.cs, s.rstd) if s.res is None else (s.y, s.c, s.cs, s.rstd, s.sum)
        fg.rmsnorm_bwd_ckpt(s.c, s.cs, s.rstd, s.w, s.dy, s.fmt, s.dx, s.dw, s.workspace, dsum=s.dsum)
        return s.dx, s.dw
    if part == "fwd":
        fg.swiglu_fwd_ckpt(s.gu, s.fmt, s.h, s.c, s.cs)
        return s.h, s.c, s.cs
    fg.swiglu_bwd_ckpt(s.c, s.cs, s.dh, s.fmt, s.dgu)
    return s.dgu


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    global own
    op, part = case["op"], case["part"]
    if op == "xent" and work(case)["flops"] > 6e12:
        return None
    was, own = own, False
    s = prepare(case, seed)
    own = was
    if op == "xent":
        # by pieces of the vocabulary: log of the sum, then the gradient of every piece
        T, V, sc, step = case["tokens"], case["vocab"], case["scale"], 4096
        used = torch.nonzero(s.target >= 0)[:, 0]
        x, at = s.x[used].double(), s.target[used].long()
        lse = torch.full((used.numel(),), -math.inf, dtype=torch.float64, device="cuda")
        for v in range(0, V, step):
            lse = torch.logaddexp(lse, torch.logsumexp(sc * (x @ s.w[v:v + step].double().T), 1))
        loss = lse - sc * (x * s.w[at].double()).sum(1)
        out = [torch.zeros(T, dtype=torch.float64, device="cuda").index_copy_(0, used, t) for t in (loss, lse)]
        if part == "fwd":
            return tuple(out)
        if part == "bwd":
            lse = s.lse[used].double()
        gl = s.dloss[used].double()
        gz = 0 if s.dlse is None else s.dlse[used].double()
        dx, dw = torch.zeros_like(x), []
        for v in range(0, V, step):
            w = s.w[v:v + step].double()
            z = torch.exp(sc * (x @ w.T) - lse[:, None]) * (gl + gz)[:, None]
            z -= (at[:, None] == torch.arange(v, v + w.shape[0], device="cuda")) * gl[:, None]
            dx += sc * (z @ w)
            dw.append(sc * (z.T @ x))
        dx = torch.zeros((T, case["dim"]), dtype=torch.float64, device="cuda").index_copy_(0, used, dx)
        return (dx, torch.cat(dw)) if part == "bwd" else (*out, dx, torch.cat(dw))
    if op == "embed":
        if part == "fwd":
            out = torch.zeros(s.out.shape, dtype=torch.float64, device="cuda")
            out[s.ids >= 0] = case["scale"] * s.w[s.ids[s.ids >= 0].long()].double()
            return out
        # by sorting the tokens and differences of running sums' ends: each id's rows are added by itself
        order = torch.argsort(s.ids, stable=True)
        order = order[s.ids[order] >= 0]
        ids, n = torch.unique_consecutive(s.ids[order], return_counts=True)
        sums = torch.segment_reduce(s.dout[order].double(), "sum", lengths=n, axis=0, unsafe=True)
        dw = s.dw.double() if case["accumulate"] else torch.zeros(s.dw.shape, dtype=torch.float64, device="cuda")
        dw[ids.long()] += case["scale"] * sums
        return dw
    fmax, bits, least = (448.0, 3, -6) if case["fmt"] == "e4m3" else (57344.0, 2, -14)

    def kept(x):    # codes, rounded to their steps, and scales
        x = x.double().reshape(x.shape[0], -1, 128)
        top = x.abs().max(2).values
        sc = torch.where(top > 0, top / fmax, 1.0)
        q = (x / sc[:, :, None]).reshape(x.shape[0], -1)
        step = torch.exp2(torch.frexp(q).exponent.clamp(min=least + 1) - 1.0 - bits)
        return torch.round(q / step) * step, sc.T

    if op == "norm":
        w = s.w.double()
        if part == "fwd":
            h = s.x if s.res is None else (s.x.double() + s.res.double()).bfloat16()
            x = h.double()
            r = ((x * x).sum(1) / case["cols"] + s.eps) ** -0.5
            y = torch.einsum("rc,r,c->rc", x, r, w)
            return (y, *kept(h), r) if s.res is None else (y, *kept(h), r, x)
        x = s.c.double() * s.cs.double().T.repeat_interleave(128, 1)
        r, dy = s.rstd.double()[:, None], s.dy.double()
        mean = torch.einsum("rc,rc,c->r", dy, x, w)[:, None] / case["cols"]
        dx = r * w * dy - r ** 3 * mean * x
        return dx if s.dsum is None else dx + s.dsum.double(), torch.einsum("rc,rc,r->c", dy, x, r[:, 0])
    F = case["ffn"]
    if part == "fwd":
        x = s.gu.double()
        return (x[:, :F] * torch.sigmoid(x[:, :F]) * x[:, F:], *kept(s.gu))
    x = s.c.double() * s.cs.double().T.repeat_interleave(128, 1)
    g, u, d = x[:, :F], x[:, F:], s.dh.double()
    t = torch.sigmoid(g)
    return torch.cat([d * u * (t + g * t * (1 - t)), d * g * t], 1)
