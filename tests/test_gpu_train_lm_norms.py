"""The training example's norms: their weights' gradients, from what reaches them and through the whole chain, and that
the optimizer applies them."""
import pytest
import torch

import fp8_fine_grained_x128_gb300 as fg
from test_gpu_train_lm import lm, off, reference

pytestmark = pytest.mark.gpu

V, D, F, T, BLOCKS = 1000, 256, 384, 384, 2


def step():
    model = lm.Model(V, D, F, blocks=BLOCKS, seed=4)
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    target = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    target[::7] = -1
    model.forward(ids, target)
    model.backward()
    assert fg.device_status() == fg.OK
    return model, ids, target


def norms(model):
    return [b.norm for b in model.blocks] + [model.norm]


def test_each_from_what_reaches_it(monkeypatch):
    """dw = sum over rows of dy n, n = codes * scales * rstd: two roundings for n, one for the product, one an addition."""
    calls, real = [], fg.rmsnorm_bwd_ckpt

    def spy(c, cs, rstd, w, dy, fmt, dx, dw, workspace, **more):
        n = (c.view(torch.float8_e4m3fn).double().unflatten(1, (-1, 128)) * cs.T.double()[..., None]).flatten(1) * rstd.double()[:, None]
        terms = dy.double() * n
        real(c, cs, rstd, w, dy, fmt, dx, dw, workspace, **more)
        calls.append((dw, dw.clone(), terms.sum(0), terms.abs().sum(0)))

    monkeypatch.setattr(fg, "rmsnorm_bwd_ckpt", spy)
    model, _, _ = step()
    assert [c[0].data_ptr() for c in calls] == [n.grad.data_ptr() for n in reversed(norms(model))]
    for dw, have, want, size in calls:
        assert float(want.abs().max()) > 0 and torch.equal(dw, have)
        assert bool(((have.double() - want).abs() <= (T + 4) * 2.0 ** -24 * size).all())


def test_gradients_through_the_chain():
    """An E4M3 rounding is off by at most 2^-4 of a value, 2^-4 / sqrt(3) in the root of the mean square, and the
    roundings of different values are independent: they add up as squares do.  A block has 12 of them on the way there
    and back (both operands of four products, twice what is kept of the norm and of SwiGLU); SwiGLU's slopes at most
    double one.  So a missing gradient (off by 1), or one scaled by 1.4, is found."""
    model, ids, target = step()
    _, ref_table, mats, ref_last = reference(model, ids, target)
    most = 2 * (12 * BLOCKS) ** 0.5 * 2.0 ** -4 / 3 ** 0.5
    assert most < 0.36
    pairs = [(model.table.grad, ref_table), (model.norm.grad, ref_last)]
    for b, (up, down, w) in zip(model.blocks, mats):
        pairs += [(b.up.grad, up.grad), (b.down.grad, down.grad), (b.norm.grad, w.grad)]
    for mine, ref in pairs:
        assert off(mine, ref) <= most
        assert float((mine.double() * ref).sum()) >= (1 - most ** 2 / 2) * float(mine.double().norm() * ref.norm())


def test_update_moves_the_norms():
    """AdamW's first step: m / bc1 = g and v / bc2 = g^2 but for a few roundings to FP32, so a weight moves by
    lr |g| / (|g| + eps) against its gradient's sign (norms have no decay); then its BF16 copy is rounded, by half a
    step of 2^-7 at most."""
    model, _, _ = step()
    lr = 2.0 ** -4
    grads = [n.grad.clone() for n in norms(model)]
    model.update(lr, 1)
    assert fg.device_status() == fg.OK
    for n, grad in zip(norms(model), grads):
        g = grad.bfloat16().double()
        assert bool((g != 0).any())
        want = -lr * g / (g.abs() + 1e-8)
        assert bool((n.w.double() - 1 - want).abs().max() <= 2.0 ** -8 + 2.0 ** -18)
