"""Linear cross entropy where nothing but the target is left of a row's logits, and sums over many tokens."""
import math

import pytest
import torch

import fp8_fine_grained_x128_gb300 as fg

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8      # half a step of BF16, relative


def forward(x, w, t, scale=1.0):
    T = x.shape[0]
    loss, lse = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    fg.linear_xent_fwd(x, w, t, loss, lse, fg.new_linear_xent_workspace(T, w.shape[0], x.shape[1]), scale=scale)
    assert fg.device_status() == fg.OK
    return loss, lse


# tokens: the one-pass forms (1, 4), single CTAs' tiles (5, 100), pairs' (300)
@pytest.mark.parametrize("T", [1, 4, 5, 100, 300])
@pytest.mark.parametrize("z", [-1000.0, -100.0, -60.0, 0.0, 60.0, 100.0])
def test_one_word(T, z):
    """A vocabulary of one word: its probability is 1, its loss 0 and lse its logit, however far that is from 0.  Sums of
    64 equal multiples of 1/64 are exact in FP32; the gradient of a row is dlse alone."""
    D = 64
    x, w = torch.ones((T, D), dtype=torch.bfloat16, device="cuda"), torch.full((1, D), z / D, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(T, dtype=torch.int32, device="cuda")
    loss, lse = forward(x, w, t)
    assert bool((loss == 0).all()) and bool((lse == z).all())
    dl, dz = torch.rand(T, device="cuda") + 0.5, torch.rand(T, device="cuda") + 0.5
    dx, dw = torch.full_like(x, 3.0), torch.full((1, D), 3.0, device="cuda")
    fg.linear_xent_bwd(x, w, t, loss, lse, dl, dx, dw, fg.new_linear_xent_workspace(T, 1, D), dlse=dz)
    assert fg.device_status() == fg.OK
    want = dz.double()[:, None] * w.double()
    assert bool(((dx.double() - want).abs() <= HALF * (1 + HALF) * want.abs()).all())      # the result's rounding
    size = float(dz.double().sum())     # a sum of x times dlse, rounded to BF16 each, in steps of 16
    assert bool(((dw.double() - size).abs() <= (HALF + (T / 16 + 16) * 2.0 ** -23) * size).all())


@pytest.mark.parametrize("T", [1, 4, 5, 100, 300])
@pytest.mark.parametrize("z", [-1000.0, -100.0, 60.0])
def test_the_other_words_ruled_out(T, z):
    """Logits of -Inf for every word but the target."""
    V, D = 5, 64
    x = torch.ones((T, D), dtype=torch.bfloat16, device="cuda")
    w = torch.full((V, D), -math.inf, dtype=torch.bfloat16, device="cuda")
    w[2] = z / D
    loss, lse = forward(x, w, torch.full((T,), 2, dtype=torch.int32, device="cuda"))
    assert bool((loss == 0).all()) and bool((lse == z).all())
    # the target ruled out, one other word left; then no word at all: the logarithm of 0, and a loss that is not a number
    loss, lse = forward(x, w, torch.full((T,), 3, dtype=torch.int32, device="cuda"))
    assert bool((loss == math.inf).all()) and bool(((lse - z).abs() <= 2.0 ** -22 * abs(z)).all())
    w[2] = -math.inf
    loss, lse = forward(x, w, torch.full((T,), 2, dtype=torch.int32, device="cuda"))
    assert bool((lse == -math.inf).all()) and bool(torch.isnan(loss).all())


@pytest.mark.parametrize("T", [2048, 16384, 65536])
@pytest.mark.parametrize("accumulate", [False, True])
def test_sums_over_many_tokens_do_not_lean(T, accumulate):
    """dw of words of equal probability 2^-8 and dlse = 1: sums of x / 256, whose terms are exact BF16 values of one sign
    (of several sizes: equal ones' sums would be exact in FP32).  2048 tokens in steps of 16, each off by at most a last
    place; the parts added to nearest."""
    V, D = 256, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.exp2(-10 * torch.rand((T, D), generator=g, device="cuda")).bfloat16()
    w = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    t = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    loss, lse = forward(x, w, t)
    dx, dw = torch.empty_like(x), torch.zeros((V, D), device="cuda")
    fg.linear_xent_bwd(x, w, t, loss, lse, torch.zeros(T, device="cuda"), dx, dw, fg.new_linear_xent_workspace(T, V, D),
                       dlse=torch.ones(T, device="cuda"), accumulate=accumulate)
    assert fg.device_status() == fg.OK
    want = x.double().sum(0) / V
    assert float(((dw.double() - want) / want).abs().max()) <= 128 * 2.0 ** -23 + (T / 2048) * 2.0 ** -24 + 2.0 ** -23


@pytest.mark.parametrize("T,V,D", [(2, 900, 512), (70, 3000, 128), (300, 3000, 128)])
def test_gradient_on_another_stream(T, V, D):
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((T, D), (V, D)))
    t = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    dl = torch.rand(T, generator=g, device="cuda")

    def step():
        loss, lse = forward(x, w, t, D ** -0.5)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        fg.linear_xent_bwd(x, w, t, loss, lse, dl, dx, dw, fg.new_linear_xent_workspace(T, V, D), scale=D ** -0.5)
        return dx, dw

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(1000000)      # the default stream would be past this call's inputs by then
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and fg.device_status() == fg.OK
