"""RMSNorm and SwiGLU with their input kept in 8 bits: codes and scales bit for bit those of quant_1x128, the BF16 results
against 64 bits from the same codes.

Tolerances: a BF16 result is off by 2^-8; FP32 sums over a row or a column of n terms by n 2^-24 of the terms' absolute
sum; the sigmoid by 1e-5 (its kernel's bound); a handful of FP32 operations by 2^-24 each."""
import math

import pytest
import torch

import fp8_fine_grained_x128_gb300 as fg

pytestmark = pytest.mark.gpu

HALF, F32 = 2.0 ** -8, 2.0 ** -24
FMTS = {"e4m3": (fg.E4M3, torch.float8_e4m3fn), "e5m2": (fg.E5M2, torch.float8_e5m2)}
ROWS_COLS = [(1, 128), (7, 256), (9, 384), (130, 512), (3, 640), (65, 1024), (33, 1920), (20, 2048), (40, 2176), (700, 4096), (5, 4224),
             (1100, 8192), (3, 8320), (400, 16384)]


def kept(x, fmt):
    R, C = x.shape
    q = torch.empty((R, C), dtype=FMTS[fmt][1], device="cuda")
    s = torch.empty((C // 128, R), device="cuda")
    fg.quant_1x128(x, FMTS[fmt][0], q, s)
    return q, s


def values(q, s):
    return (q.float().double().unflatten(1, (-1, 128)) * s.double().T[..., None]).flatten(1)


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def inputs(R, C, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((R, C + 8), generator=g, device="cuda").bfloat16()[:, :C]
    res = (torch.randn((R, C + 16), generator=g, device="cuda") * 3).bfloat16()[:, :C]
    w = (1 + 0.2 * torch.randn(C, generator=g, device="cuda")).bfloat16()
    return x, res, w


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("R,C", ROWS_COLS)
def test_norm_forward(R, C, residual, fmt):
    x, res, w = inputs(R, C)
    if R > 2:
        x[1] = 0
        res[1] = 0          # a row of zeros: rstd = eps^-1/2, unit scales
    eps = 1e-5
    wide = torch.full((R + 1, C + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    y, total = wide[:R, :C], torch.empty((R, C), dtype=torch.bfloat16, device="cuda") if residual else None
    c, cs, rstd = torch.empty((R, C), dtype=torch.uint8, device="cuda"), torch.empty((C // 128, R), device="cuda"), torch.empty(R, device="cuda")
    fg.rmsnorm_fwd_ckpt(x, w, eps, FMTS[fmt][0], y, c, cs, rstd, res=res if residual else None, sum=total)
    assert fg.device_status() == fg.OK
    assert bool((wide[R:] == 3).all()) and bool((wide[:, C:] == 3).all())
    h = (x.float() + res.float()).bfloat16() if residual else x
    if residual:
        assert torch.equal(total, h)
    q, s = kept(h, fmt)
    assert same(c, q) and torch.equal(cs, s)
    X = h.double()
    want = (X.square().mean(1) + eps) ** -0.5
    # the mean is off by C 2^-24 at most, and its root's inverse by half of that and 2 ulp
    tol = (C / 2 + 8) * F32
    assert bool(((rstd - want).abs() <= tol * want).all())
    Y = X * want[:, None] * w.double()
    assert bool(((y.double() - Y).abs() <= (HALF + 1.01 * tol + 4 * F32) * Y.abs()).all())


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("R,C", ROWS_COLS)
def test_norm_backward(R, C, residual, fmt):
    x, _, w = inputs(R, C, 1)
    if R > 2:
        x[1] = 0
    c, cs = kept(x, fmt)
    rstd = (x.double().square().mean(1) + 1e-5).rsqrt().float()
    g = torch.Generator(device="cuda").manual_seed(2)
    dy = torch.randn((R, C + 8), generator=g, device="cuda").bfloat16()[:, :C]
    dsum = torch.randn((R, C + 24), generator=g, device="cuda").bfloat16()[:, :C] if residual else None
    ws = fg.new_rmsnorm_workspace(C)
    ws.fill_(255)
    wide = torch.full((R + 1, C + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(C, device="cuda")
    fg.rmsnorm_bwd_ckpt(c, cs, rstd, w, dy, FMTS[fmt][0], wide[:R, :C], dw, ws, dsum=dsum)
    assert fg.device_status() == fg.OK
    assert bool((wide[R:] == 3).all()) and bool((wide[:, C:] == 3).all())
    n = values(c, cs) * rstd.double()[:, None]
    D, W, r = dy.double(), w.double(), rstd.double()[:, None]
    t = D * W
    dot = (t * n).mean(1, keepdim=True)
    want = (t - n * dot) * r
    # the mean's C terms, then a few operations on each of the two terms and the sum
    tol = ((t.abs() + n.abs() * dot.abs()) * 8 * F32 + n.abs() * (t * n).abs().mean(1, keepdim=True) * (C + 8) * F32) * r
    if residual:
        want, tol = want + dsum.double(), tol + 2 * F32 * dsum.double().abs()
    assert bool(((wide[:R, :C].double() - want).abs() <= tol * (1 + HALF) + HALF * want.abs() + 2.0 ** -130).all())
    size = (D * n).abs().sum(0)
    assert bool(((dw - (D * n).sum(0)).abs() <= (R + 8) * F32 * size + 1e-30).all())
    # added to, and the same in every run
    more = torch.full((C,), 2.0, device="cuda")
    dx = torch.empty((R, C), dtype=torch.bfloat16, device="cuda")
    fg.rmsnorm_bwd_ckpt(c, cs, rstd, w, dy, FMTS[fmt][0], dx, more, ws, dsum=dsum, accumulate=True)
    assert torch.equal(more, dw + 2.0) and torch.equal(dx, wide[:R, :C])


def test_norm_in_place():
    R, C = 77, 1536
    x, res, w = inputs(R, C, 3)
    x, res = x.contiguous(), res.contiguous()
    c, cs, rstd = torch.empty((R, C), dtype=torch.uint8, device="cuda"), torch.empty((C // 128, R), device="cuda"), torch.empty(R, device="cuda")
    y, total = torch.empty_like(x), torch.empty_like(x)
    fg.rmsnorm_fwd_ckpt(x, w, 1e-6, fg.E4M3, y, c, cs, rstd, res=res, sum=total)
    a, b = x.clone(), res.clone()
    fg.rmsnorm_fwd_ckpt(a, w, 1e-6, fg.E4M3, a, c, cs, rstd, res=b, sum=b)
    assert torch.equal(a, y) and torch.equal(b, total)
    dy, dsum, ws = torch.randn_like(x), torch.randn_like(x), fg.new_rmsnorm_workspace(C)
    dx, dw = torch.empty_like(x), torch.empty(C, device="cuda")
    fg.rmsnorm_bwd_ckpt(c, cs, rstd, w, dy, fg.E4M3, dx, dw, ws, dsum=dsum)
    dw2 = torch.empty_like(dw)
    for i in (0, 1):
        pair = [dy.clone(), dsum.clone()]
        fg.rmsnorm_bwd_ckpt(c, cs, rstd, w, pair[0], fg.E4M3, pair[i], dw2, ws, dsum=pair[1])
        assert torch.equal(pair[i], dx) and torch.equal(dw2, dw)


def test_norm_gradient_against_differences():
    """The slope of sum(y dy) in 64 bits, at the input that the codes stand for, along the kernel's gradients."""
    R, C, eps = 30, 512, 1e-5
    x, _, w = inputs(R, C, 4)
    c, cs = kept(x, "e4m3")
    X = values(c, cs)
    rstd = (X.square().mean(1) + eps).rsqrt().float()
    dy = torch.randn((R, C), device="cuda").bfloat16()
    dx, dw = torch.empty((R, C), dtype=torch.bfloat16, device="cuda"), torch.empty(C, device="cuda")
    fg.rmsnorm_bwd_ckpt(c, cs, rstd, w, dy, fg.E4M3, dx, dw, fg.new_rmsnorm_workspace(C))

    def value(X, W):
        return (X * (X.square().mean(1, keepdim=True) + eps).rsqrt() * W * dy.double()).sum()

    for a, b in ((dx.double(), 0.0), (0.0, dw.double())):
        n = float((a if isinstance(b, float) else b).norm())
        h = 1e-4
        slope = (value(X + h * a / n, w.double() + h * b / n) - value(X - h * a / n, w.double() - h * b / n)) / (2 * h)
        assert abs(float(slope) - n) <= 2 * HALF * n


def test_norm_rows_of_none():
    C = 256
    e = torch.empty((0, C), dtype=torch.bfloat16, device="cuda")
    w, ws = torch.ones(C, dtype=torch.bfloat16, device="cuda"), fg.new_rmsnorm_workspace(C)
    z, codes = torch.empty(0, device="cuda"), torch.empty((0, C), dtype=torch.uint8, device="cuda")
    fg.rmsnorm_fwd_ckpt(e, w, 1e-5, fg.E4M3, e, codes, z, z)
    dw = torch.ones(C, device="cuda")
    fg.rmsnorm_bwd_ckpt(codes, z, z, w, e, fg.E4M3, e, dw, ws, accumulate=True)
    assert bool((dw == 1).all())
    fg.rmsnorm_bwd_ckpt(codes, z, z, w, e, fg.E4M3, e, dw, ws)
    assert not dw.any() and fg.device_status() == fg.OK


SWIGLU = [(1, 128), (3, 384), (7, 512), (8, 640), (130, 1408), (33, 2176), (300, 14336)]


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("R,F", SWIGLU)
def test_swiglu(R, F, fmt):
    g = torch.Generator(device="cuda").manual_seed(5)
    gu = (torch.randn((R, 2 * F), generator=g, device="cuda") * 3).bfloat16()
    gu[0, :64] = torch.linspace(-300, 300, 64, device="cuda").bfloat16()     # gates of the whole range
    if R > 2:
        gu[1, :128] = 0
    h, ref = (torch.empty((R, F), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c = torch.empty((R, 2 * F), dtype=FMTS[fmt][1], device="cuda")
    cs = torch.empty((2 * F // 128, R), device="cuda")
    fg.swiglu_fwd_ckpt(gu, FMTS[fmt][0], h, c, cs)
    fg.swiglu_fwd(gu, ref)
    q, s = kept(gu, fmt)
    assert fg.device_status() == fg.OK
    assert torch.equal(h, ref) and same(c, q) and torch.equal(cs, s)

    dh = torch.randn((R, F), generator=g, device="cuda").bfloat16()
    dgu = torch.full((R + 1, 2 * F), 3.0, dtype=torch.bfloat16, device="cuda")
    fg.swiglu_bwd_ckpt(c, cs, dh, FMTS[fmt][0], dgu[:R])
    assert fg.device_status() == fg.OK and bool((dgu[R:] == 3).all())
    G, U = values(c, cs).chunk(2, 1)
    D, sig = dh.double(), torch.sigmoid(G)
    want = torch.cat([D * U * (sig + G * sig * (1 - sig)), D * G * sig], 1)
    # the sigmoid enters the gate's gradient three times, once beside a difference from 1
    size = torch.cat([(D * U).abs() * sig * (1 + 2 * G.abs()), (D * G).abs() * sig], 1)
    assert bool(((dgu[:R].double() - want).abs() <= HALF * want.abs() + 3e-5 * size + 2.0 ** -126).all())


def test_nonfinite_is_recorded():
    for bad in (math.nan, math.inf):
        x = torch.randn((5, 256), device="cuda").bfloat16()
        x[3, 200] = bad
        c, cs, rstd = torch.empty((5, 256), dtype=torch.uint8, device="cuda"), torch.empty((2, 5), device="cuda"), torch.empty(5, device="cuda")
        y = torch.empty_like(x)
        fg.rmsnorm_fwd_ckpt(x, torch.ones(256, dtype=torch.bfloat16, device="cuda"), 1e-5, fg.E4M3, y, c, cs, rstd)
        assert fg.device_status() == fg.ERR_NONFINITE
        fg.swiglu_fwd_ckpt(x, fg.E4M3, torch.empty((5, 128), dtype=torch.bfloat16, device="cuda"), c, cs)
        assert fg.device_status() == fg.ERR_NONFINITE


def test_columns_that_are_no_pair_are_refused():
    gu, h = torch.zeros((2, 257), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        fg.swiglu_fwd_ckpt(gu, fg.E4M3, h, torch.zeros((2, 257), dtype=torch.uint8, device="cuda"), torch.zeros((2, 2), device="cuda"))


@pytest.mark.parametrize("R,C", [(5, 512), (900, 2048)])
def test_captured_on_another_stream(R, C):
    """Norm and SwiGLU, forward and backward, as one graph of their own stream, replayed with other inputs."""
    x, res, w = inputs(R, C, 31)
    x2, res2, _ = inputs(R, C, 32)
    side, F = torch.cuda.Stream(), C // 2
    bf = lambda cols: torch.empty((R, cols), dtype=torch.bfloat16, device="cuda")
    y, total, h, dgu, dx, c, cs = bf(C), bf(C), bf(F), bf(C), bf(C), torch.empty((R, C), dtype=torch.uint8, device="cuda"), torch.empty((C // 128, R), device="cuda")
    c2, cs2, rstd, dw, ws = torch.empty_like(c), torch.empty_like(cs), torch.empty(R, device="cuda"), torch.zeros(C, device="cuda"), fg.new_rmsnorm_workspace(C)

    def step():
        fg.rmsnorm_fwd_ckpt(x, w, 1e-5, fg.E4M3, y, c, cs, rstd, res=res, sum=total)
        fg.swiglu_fwd_ckpt(y, fg.E5M2, h, c2, cs2)
        fg.swiglu_bwd_ckpt(c2, cs2, h, fg.E5M2, dgu)
        fg.rmsnorm_bwd_ckpt(c, cs, rstd, w, dgu, fg.E4M3, dx, dw, ws, dsum=total)
        return [a.clone() for a in (y, total, h, dgu, dx, dw, c, c2)]

    want = []
    for a, b in ((x, res), (x2, res2)):
        x, res = a, b
        want.append(step())
    first = inputs(R, C, 31)
    x, res = (a.clone() for a in first[:2])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
    for (a, b), ref in zip((first[:2], (x2, res2)), want):
        x.copy_(a)
        res.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(m, n) for m, n in zip(got, ref)) and fg.device_status() == fg.OK


def test_offsets_beyond_32_bits_full_size():
    """More than 2^31 elements: the last rows are as those of a small call."""
    R, F = 90000, 14336
    gu = torch.empty((R, 2 * F), dtype=torch.bfloat16, device="cuda").normal_()
    h, c, cs = torch.empty((R, F), dtype=torch.bfloat16, device="cuda"), torch.empty((R, 2 * F), dtype=torch.uint8, device="cuda"), torch.empty((2 * F // 128, R), device="cuda")
    fg.swiglu_fwd_ckpt(gu, fg.E4M3, h, c, cs)
    dgu = torch.empty_like(gu)
    fg.swiglu_bwd_ckpt(c, cs, h, fg.E4M3, dgu)
    n = 300
    last = gu[-n:].contiguous()
    h2, c2, cs2, d2 = torch.empty((n, F), dtype=torch.bfloat16, device="cuda"), torch.empty((n, 2 * F), dtype=torch.uint8, device="cuda"), torch.empty((2 * F // 128, n), device="cuda"), torch.empty_like(last)
    fg.swiglu_fwd_ckpt(last, fg.E4M3, h2, c2, cs2)
    fg.swiglu_bwd_ckpt(c2, cs2, h2, fg.E4M3, d2)
    assert torch.equal(h[-n:], h2) and torch.equal(c[-n:], c2) and torch.equal(cs[:, -n:], cs2) and torch.equal(dgu[-n:], d2)
    del h, c, cs, dgu
    R, C = 140000, 16384
    x = gu.view(-1)[:R * C].view(R, C)
    w, ws = torch.randn(C, device="cuda").bfloat16(), fg.new_rmsnorm_workspace(C)

    def both(x):
        R = x.shape[0]
        y, c, cs, r = torch.empty_like(x), torch.empty((R, C), dtype=torch.uint8, device="cuda"), torch.empty((C // 128, R), device="cuda"), torch.empty(R, device="cuda")
        fg.rmsnorm_fwd_ckpt(x, w, 1e-5, fg.E4M3, y, c, cs, r)
        dx, dw = torch.empty_like(x), torch.empty(C, device="cuda")
        fg.rmsnorm_bwd_ckpt(c, cs, r, w, y, fg.E4M3, dx, dw, ws)
        return y, c, r, dx

    big, small = both(x), both(x[-n:].contiguous())
    assert all(torch.equal(a[-n:], b) for a, b in zip(big, small)) and fg.device_status() == fg.OK
