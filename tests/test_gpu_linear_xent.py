"""Linear cross entropy against its definition in 64 bits: sizes around the kernels' tiles, tokens that do not count,
strided operands, both gradients' types, and what each must leave alone.

Tolerances, from the arithmetic alone.  A logit is a sum of D exact products in FP32, 16 a step, each step and each
addition inside it off by at most 2^-23 of the terms' sum A = sum |x w|: off = (D / 16 + 16) 2^-23 A.  The sum of
exponentials: 2^-22 an exponential, 2^-23 of its argument, and one rounding for each of the at most V / 32 + 40
additions on a term's way.  The rows of g, relative to the target's entry, are rounded to BF16 (2^-8 at most; the
target's own entry not), for dw also x times that entry, and so are BF16 results."""
import math

import pytest
import torch

import fp8_fine_grained_x128_gb300 as fg

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8      # half a step of BF16, relative


def make(T, V, D, ignored=0.0, seed=0, lift=8.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn((V, D + pad), generator=g, device="cuda") * 1.5 * D ** -0.5).bfloat16()[:, :D]
    t = torch.randint(V, (T,), generator=g, device="cuda")
    x = torch.randn((T, D + pad), generator=g, device="cuda").bfloat16()
    x[:, :D] += (torch.rand((T, 1), generator=g, device="cuda") * lift / 2.25 * w[t].float()).bfloat16()
    t[torch.rand(T, generator=g, device="cuda") < ignored] = -100
    return x[:, :D], w, t.to(torch.int32)


def exact(x, w, t, scale):
    z = scale * (x.double() @ w.double().T)
    lse = torch.logsumexp(z, 1)
    at = t.clamp(min=0).long()[:, None]
    rest = z.scatter(1, at, -math.inf)
    rest = torch.logsumexp(rest, 1) - z.gather(1, at)[:, 0]      # log of the rest's sum relative to the target
    loss = torch.nn.functional.softplus(rest, threshold=100.0)
    if z.shape[1] == 1:
        loss = torch.zeros_like(lse)
    return z, lse, loss


def logit_error(x, w, scale):
    D = x.shape[1]
    return (D / 16 + 16) * 2.0 ** -23 * scale * float((x.double().abs() @ w.double().abs().T).max())


def sum_error(V, z):
    return (V / 32 + 40) * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -22 * float(z.abs().max())


def forward(x, w, t, scale=1.0, ws=None):
    T = x.shape[0]
    loss, lse = torch.full((T + 8,), 7.0, device="cuda"), torch.full((T + 8,), 7.0, device="cuda")
    if ws is None:
        ws = fg.new_linear_xent_workspace(T, w.shape[0], x.shape[1])
    fg.linear_xent_fwd(x, w, t, loss[:T], lse[:T], ws, scale=scale)
    assert fg.device_status() == fg.OK
    assert bool((loss[T:] == 7).all()) and bool((lse[T:] == 7).all())
    return loss[:T], lse[:T]


SIZES = [(1, 1, 8), (1, 257, 64), (2, 7, 8), (3, 5003, 72), (127, 256, 128), (128, 255, 200), (129, 1000, 64), (255, 513, 136),
         (256, 256, 256), (257, 1025, 64), (300, 2000, 512), (513, 300, 1024), (1000, 9001, 320), (5, 40000, 1024), (4, 10007, 1032), (2, 31, 4096), (1, 70001, 8), (4, 300, 8192), (70, 400, 6152),
         (1, 5001, 3992), (2, 3001, 264), (3, 2002, 4096), (40, 470000, 8)]


@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("ignored,scale,pad", [(0.0, 1.0, 0), (0.4, 0.3, 24)])
def test_forward(T, V, D, ignored, scale, pad):
    x, w, t = make(T, V, D, ignored, seed=T + V + D, pad=pad)
    loss, lse = forward(x, w, t, scale)
    z, want_lse, want = exact(x, w, t, scale)
    counts = t >= 0
    tol = logit_error(x, w, scale) + sum_error(V, z)
    assert bool(((lse - want_lse).abs()[counts] <= tol + 2.0 ** -22 * want_lse.abs()[counts]).all())
    assert bool(((loss - want).abs()[counts] <= 2 * tol + 2.0 ** -22 * want.abs()[counts]).all())
    assert bool((loss[~counts] == 0).all()) and bool((lse[~counts] == 0).all())


def test_small_losses_keep_their_digits():
    """Tokens predicted with 12 to 60 on the target's logit: the loss is relatively as exact as the logits' differences are."""
    T, V, D = 64, 3000, 256
    x, w, t = make(T, V, D, seed=3, lift=0.0)
    x = (torch.linspace(12, 60, T, device="cuda")[:, None] / 2.25 * w[t.long()].float()).bfloat16()
    loss, lse = forward(x, w, t)
    z, _, want = exact(x, w, t, 1.0)
    tol = 2 * logit_error(x, w, 1.0) + 2 * sum_error(V, z) + 2.0 ** -20
    assert float(want.min()) < 1e-15
    normal = want > 2.0 ** -125
    assert bool(((loss - want).abs() <= want * tol)[normal].all())


@pytest.mark.parametrize("T", [4, 40, 700])
def test_rows_that_do_not_count_hold_anything(T):
    x, w, t = make(T, 900, 128, 0.5, seed=5)
    dl, dz = torch.rand(T, device="cuda"), torch.rand(T, device="cuda")
    clean = [a.clone() for a in forward(x, w, t)]
    dx, dw = backward(x, w, t, *clean, dl, dz)
    out = t < 0
    for bad in (math.nan, math.inf):
        x[out] = bad
        dl[out] = bad
        dz[out] = bad
        again = forward(x, w, t)
        assert all(torch.equal(a, b) for a, b in zip(clean, again))
        dx2, dw2 = backward(x, w, t, *again, dl, dz)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    assert bool((dx[out] == 0).all())


@pytest.mark.parametrize("T", [3, 400])
def test_a_nan_row_stays_its_own(T):
    x, w, t = make(T, 700, 64, seed=6)
    loss, lse = forward(x, w, t)
    x[1, 5] = math.nan
    loss2, lse2 = forward(x, w, t)
    keep = torch.arange(T, device="cuda") != 1
    assert torch.equal(loss[keep], loss2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert math.isnan(loss2[1]) and math.isnan(lse2[1])


def test_no_token_counts():
    for T in (1, 200, 600):
        x, w, t = make(T, 500, 64, seed=7)
        t.fill_(-1)
        loss, lse = forward(x, w, t)
        assert not loss.any() and not lse.any()
        dx, dw = backward(x, w, t, loss, lse, torch.ones(T, device="cuda"), None)
        assert not dx.any() and not dw.any()
        base = torch.randn((500, 64), device="cuda")
        dw32 = base.clone()
        backward(x, w, t, loss, lse, torch.ones(T, device="cuda"), None, dw=dw32, accumulate=True)
        assert torch.equal(dw32, base)


def test_target_out_of_range_is_recorded_and_left_out():
    for T in (4, 30, 300):
        x, w, t = make(T, 100, 64, seed=8)
        ref = t.clone()
        ref[[2, T - 1]] = -1
        t[2], t[T - 1] = 100, 1 << 30
        ws = fg.new_linear_xent_workspace(T, 100, 64)
        loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        fg.linear_xent_fwd(x, w, t, loss, lse, ws)
        assert fg.device_status() == fg.ERR_INVALID_ARG
        want = forward(x, w, ref)
        assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])
        dl = torch.ones(T, device="cuda")
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        fg.linear_xent_bwd(x, w, t, loss, lse, dl, dx, dw, ws)
        assert fg.device_status() == fg.ERR_INVALID_ARG
        dx2, dw2 = backward(x, w, ref, *want, dl, None)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def backward(x, w, t, loss, lse, dloss, dlse, scale=1.0, dw=None, accumulate=False, ws=None):
    T, D = x.shape
    V = w.shape[0]
    dx = torch.full((T + 2, D + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    if dw is None:
        dw = torch.full((V, D), 3.0, dtype=torch.bfloat16, device="cuda")
    if ws is None:
        ws = fg.new_linear_xent_workspace(T, V, D)
    fg.linear_xent_bwd(x, w, t, loss, lse, dloss, dx[:T, :D], dw, ws, dlse=dlse, scale=scale, accumulate=accumulate)
    assert fg.device_status() == fg.OK
    assert bool((dx[T:] == 3).all()) and bool((dx[:, D:] == 3).all())
    return dx[:T, :D], dw


@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("ignored,scale,pad,zloss,kind", [(0.0, 1.0, 0, False, "bf16"), (0.4, 0.3, 24, True, "f32"), (0.2, 1.0, 8, True, "add")])
def test_gradients(T, V, D, ignored, scale, pad, zloss, kind):
    x, w, t = make(T, V, D, ignored, seed=T + V + D + 1, pad=pad)
    g = torch.Generator(device="cuda").manual_seed(9)
    dl = (torch.rand(T, generator=g, device="cuda") + 0.5) / T
    dz = torch.randn(T, generator=g, device="cuda") / T if zloss else None
    loss, lse = forward(x, w, t, scale)
    wide = torch.full((V + 1, D + 8), 2.0, dtype=torch.bfloat16 if kind == "bf16" else torch.float32, device="cuda")
    base = torch.randn((V, D), generator=g, device="cuda") / T if kind == "add" else None
    if base is not None:
        wide[:V, :D] = base
    dx, dw = backward(x, w, t, loss, lse, dl, dz, scale, dw=wide[:V, :D], accumulate=kind == "add")
    assert bool((wide[V:] == 2).all()) and bool((wide[:, D:] == 2).all())

    z, want_lse, want_loss = exact(x, w, t, scale)
    counts = (t >= 0)[:, None]
    gl = torch.where(counts, dl.double()[:, None], 0)
    gz = torch.where(counts, dz.double()[:, None], 0) if zloss else torch.zeros_like(gl)
    p = torch.exp(z - want_lse[:, None])
    at = torch.nn.functional.one_hot(t.clamp(min=0).long(), V).double()
    pm = torch.where(at > 0, torch.expm1(-want_loss)[:, None], p)        # p - [v = target]
    G = scale * (gl * pm + gz * p)
    size = scale * (gl.abs() * pm.abs() + gz.abs() * p)                   # what the rounding of g's terms goes by
    # p: its logit's error and lse's (which holds the same), the exponential's, a division; then g's rounding and, for
    # dw, that of x times the entry, whose product a term is
    off = 2 * (logit_error(x, w, scale) + sum_error(V, z)) + 2.0 ** -20 + 2.0 ** -22 * float(want_lse.abs().max())
    rel = HALF + off * 1.01
    X, W = x.double(), w.double()
    X = torch.where(counts, X, 0)
    want_dx, want_dw = G @ W, G.T @ X
    tol_dx = rel * (size @ W.abs()) + (V / 16 + 64) * 2.0 ** -23 * (size @ W.abs())
    tol_dw = (rel + HALF * (1 + HALF)) * (size.T @ X.abs()) + (T / 16 + 64) * 2.0 ** -23 * (size.T @ X.abs())
    tiny = 2.0 ** -126
    assert bool(((dx.double() - want_dx).abs() <= tol_dx * (1 + HALF) + HALF * want_dx.abs() + tiny).all())
    have = dw.double()
    if base is not None:
        want_dw = want_dw + base.double()
        tol_dw = tol_dw + 2.0 ** -23 * want_dw.abs() + 2.0 ** -24 * base.double().abs()
    assert bool(((have - want_dw).abs() <= tol_dw * (1 + HALF) + (HALF if kind == "bf16" else 0) * want_dw.abs() + tiny).all())
    # over many values the roundings do not add up: their root mean square is below half a step each
    if T * D > 4000 and bool(counts.any()):
        assert float((dx.double() - want_dx).norm()) <= (2 * HALF + off) * float(want_dx.norm())


@pytest.mark.parametrize("gl,gz", [(0.0, 2.0 ** 30), (0.0, 1.0), (-(2.0 ** -90), 2.0 ** 30), (2.0 ** 30, 0.0)])
@pytest.mark.parametrize("at", [-89.4, -60.0, 89.4, 60.0])
def test_entries_far_from_the_targets(gl, gz, at):
    """A target at 1e-39 (or at 1 but for 1e-39) of the probability: its entry and the others' are far apart, and no
    quotient of them may leave the range of FP32.  Every term is off by at most two roundings to BF16, those of p's
    exponent (2^-15 of it at 93) and the result's; probabilities below 2^-126 may count as zero, V of them in the loss."""
    T, V, D = 5, 40, 64
    u = torch.linspace(0.5, 1.0, D, device="cuda").bfloat16()
    w = torch.zeros((V, D), device="cuda")
    w[3] = (at + math.log(V)) / float(u.double() @ u.double()) * u.float()
    w[7, 5] = w[9, 6] = 0.25
    w, x, t = w.bfloat16(), u.repeat(T, 1), torch.full((T,), 3, dtype=torch.int32, device="cuda")
    loss, lse = forward(x, w, t)
    dx, dw = backward(x, w, t, loss, lse, torch.full((T,), gl, device="cuda"), torch.full((T,), gz, device="cuda"),
                      dw=torch.empty((V, D), device="cuda"))
    z, _, want_loss = exact(x, w, t, 1.0)
    p = torch.softmax(z, 1)
    G = (gl + gz) * p
    G[:, 3] = (gl * torch.expm1(-want_loss) + gz * torch.exp(-want_loss))
    for have, want, terms in ((dx, G @ w.double(), G.abs() @ w.double().abs()), (dw, G.T @ x.double(), G.abs().T @ x.double().abs())):
        assert bool(torch.isfinite(have).all())
        flush = (abs(gl) + abs(gz)) * V * 2.0 ** -126 * V * float(w.double().abs().max())
        assert bool(((have.double() - want).abs() <= 4 * HALF * terms + flush + 2.0 ** -126).all())


def test_gradient_against_differences():
    """The directional derivative of the forward in 64 bits along the kernel's own gradients."""
    T, V, D = 48, 333, 64
    x, w, t = make(T, V, D, 0.25, seed=11)
    dl, dz = torch.rand(T, device="cuda") / T, torch.rand(T, device="cuda") / T
    loss, lse = forward(x, w, t)
    dx, dw = backward(x, w, t, loss, lse, dl, dz)

    def value(X, W):
        z = X @ W.T
        lse = torch.logsumexp(z, 1)
        at = z.gather(1, t.clamp(min=0).long()[:, None])[:, 0]
        return torch.where(t >= 0, dl.double() * (lse - at) + dz.double() * lse, 0).sum()

    X, W, h = x.double(), w.double(), 1e-4
    for a, b in ((dx.double(), 0 * W), (0 * X, dw.double())):
        n = float((a.square().sum() + b.square().sum()).sqrt())
        a, b = a / n, b / n
        slope = (value(X + h * a, W + h * b) - value(X - h * a, W - h * b)) / (2 * h)
        # along its own direction a gradient's slope is its norm; g's and the result's roundings, and h^2
        assert abs(float(slope) - n) <= 2 * HALF * n + 1e-6


def test_many_pieces_of_the_vocabulary():
    """More tokens than one piece of the vocabulary has room for: dx is summed over pieces, each writes its part of dw."""
    T, V, D = 16400, 24600, 64      # 112M / 16640 rows -> pieces of 6912 at most: four of them
    x, w, t = make(T, V, D, 0.1, seed=12)
    dl = torch.full((T,), 1.0 / T, device="cuda")
    loss, lse = forward(x, w, t)
    dx, dw = backward(x, w, t, loss, lse, dl, None)
    rows = torch.cat([torch.arange(200, device="cuda"), torch.arange(T - 200, T, device="cuda")])
    z, want_lse, want = exact(x[rows], w, t[rows], 1.0)
    counts = (t[rows] >= 0)[:, None]
    G = torch.where(counts, (torch.exp(z - want_lse[:, None]) - torch.nn.functional.one_hot(t[rows].clamp(min=0).long(), V)) / T, 0)
    ref = G @ w.double()
    assert float((dx[rows].double() - ref).norm()) <= 2 * HALF * float(ref.norm())
    ref = torch.zeros((V, D), dtype=torch.float64, device="cuda")
    for r in range(0, T, 2048):
        z = x[r:r + 2048].double() @ w.double().T
        p = torch.softmax(z, 1)
        tt = t[r:r + 2048]
        p[torch.arange(tt.numel(), device="cuda"), tt.clamp(min=0).long()] -= 1
        ref += torch.where((tt >= 0)[:, None], p / T, 0).T @ x[r:r + 2048].double()
    assert float((dw.double() - ref).norm()) <= 2 * HALF * float(ref.norm())


def test_runs_repeat_and_graphs_replay():
    T, V, D = 500, 4000, 256
    x, w, t = make(T, V, D, 0.3, seed=13)
    dl = torch.rand(T, device="cuda")
    ws = fg.new_linear_xent_workspace(T, V, D)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)

    def step():
        fg.linear_xent_fwd(x, w, t, loss, lse, ws)
        fg.linear_xent_bwd(x, w, t, loss, lse, dl, dx, dw, ws)

    step()
    first = [a.clone() for a in (loss, lse, dx, dw)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for a in (loss, lse, dx, dw):
        a.fill_(5)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, (loss, lse, dx, dw)))
    # other tokens, more of them counted, in the same buffers: the graph reads them on the device
    x2, _, t2 = make(T, V, D, 0.0, seed=14)
    x.copy_(x2)
    t.copy_(t2)
    graph.replay()
    got = [a.clone() for a in (loss, lse, dx, dw)]
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, (loss, lse, dx, dw)))
    assert fg.device_status() == fg.OK


def test_one_workspace_for_calls_of_many_sizes():
    ws = fg.new_linear_xent_workspace(1000, 5000, 520)
    for T, V, D in ((1000, 5000, 64), (1000, 300, 520), (2, 5000, 520), (100, 4999, 512), (257, 700, 136)):
        x, w, t = make(T, V, D, 0.2, seed=T)
        own = forward(x, w, t)
        shared = forward(x, w, t, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(own, shared))
        dl = torch.rand(T, device="cuda")
        for a, b in zip(backward(x, w, t, *own, dl, None), backward(x, w, t, *own, dl, None, ws=ws)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,V,D", [(1, 3000, 640), (4, 2000, 264), (2, 900, 4096), (30, 3000, 328), (200, 1500, 256)])
def test_small_calls_replay(T, V, D):
    """The forms for few tokens and few tiles, captured and replayed with other inputs, two calls behind one another."""
    x, w, t = make(T, V, D, seed=T)
    x2, w2, t2 = (a.contiguous() for a in make(T, V, D, 0.5, seed=T + 1))
    x, w, dl = x.contiguous(), w.contiguous(), torch.rand(T, device="cuda")
    ws, loss, lse = fg.new_linear_xent_workspace(T, V, D), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dx, dw = torch.empty_like(x), torch.zeros((V, D), device="cuda")

    def step():
        for _ in range(2):
            fg.linear_xent_fwd(x, w, t, loss, lse, ws)
            fg.linear_xent_bwd(x, w, t, loss, lse, dl, dx, dw, ws, accumulate=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for a, b in ((x, x2), (w, w2), (t, t2)):
        a.copy_(b)
    dw.zero_()
    graph.replay()
    got = [a.clone() for a in (loss, lse, dx, dw)]
    dw.zero_()
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, (loss, lse, dx, dw))) and fg.device_status() == fg.OK


def test_gradient_in_place():
    """dx may be x: every row of it has been copied before any is written."""
    for T in (3, 100, 700):
        x, w, t = make(T, 1000, 128, 0.3, seed=16)
        dl = torch.rand(T, device="cuda")
        loss, lse = forward(x, w, t)
        dx, dw = backward(x, w, t, loss, lse, dl, None)
        ws, again = fg.new_linear_xent_workspace(T, 1000, 128), torch.empty_like(w)
        fg.linear_xent_bwd(x, w, t, loss, lse, dl, x, again, ws)
        assert torch.equal(x, dx) and torch.equal(again, dw) and fg.device_status() == fg.OK


def test_on_another_stream():
    x, w, t = make(300, 3000, 128, seed=15)
    want = forward(x, w, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = fg.new_linear_xent_workspace(300, 3000, 128)
        loss, lse = torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
        fg.linear_xent_fwd(x, w, t, loss, lse, ws)
    s.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])


def test_no_tokens():
    w = torch.randn((10, 64), device="cuda").bfloat16()
    x, e = w[:0], torch.empty(0, device="cuda")
    t = torch.empty(0, dtype=torch.int32, device="cuda")
    ws = fg.new_linear_xent_workspace(0, 10, 64)
    fg.linear_xent_fwd(x, w, t, e, e, ws)
    dw = torch.ones((10, 64), device="cuda")
    fg.linear_xent_bwd(x, w, t, e, e, e, x, dw, ws, accumulate=True)
    assert bool((dw == 1).all())
    fg.linear_xent_bwd(x, w, t, e, e, e, x, dw, ws)
    assert not dw.any()


@pytest.mark.parametrize("T,V,D", [(3, 270000, 8192), (40, 270000, 8192), (300, 270000, 8192), (2, 540000, 4096)])
def test_offsets_beyond_32_bits_full_size(T, V, D):
    """W and dw of more than 2^31 elements: targets at both ends, checked on slices of the vocabulary."""
    g = torch.Generator(device="cuda").manual_seed(17)
    w = torch.empty((V, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g).mul_(D ** -0.5)
    x = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    t = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    t[0], t[1] = V - 1, 0
    x[0] += 20 * w[V - 1]
    loss, lse = forward(x, w, t)
    z = torch.cat([x.double() @ w[v:v + 30000].double().T for v in range(0, V, 30000)], 1)
    want = torch.logsumexp(z, 1)
    at = z.gather(1, t.long()[:, None])[:, 0]
    off = (D / 16 + 16) * 2.0 ** -23 * float((x.double().abs() @ w[:2000].double().abs().T).max()) * 1.5 + sum_error(V, z)
    assert float((lse - want).abs().max()) <= off and float((loss - (want - at)).abs().max()) <= 2 * off
    dl = torch.ones(T, device="cuda")
    dx, dw = backward(x, w, t, loss, lse, dl, None)
    p = torch.exp(z - want[:, None])
    p[torch.arange(T, device="cuda"), t.long()] -= 1
    ref = sum(p[:, v:v + 30000] @ w[v:v + 30000].double() for v in range(0, V, 30000))
    assert float((dx.double() - ref).norm()) <= 2 * HALF * float(ref.norm())
    for v in (0, V // 2, V - 500):
        ref = p[:, v:v + 500].T @ x.double()
        assert float((dw[v:v + 500].double() - ref).norm()) <= 2 * HALF * float(ref.norm())
