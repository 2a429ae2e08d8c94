"""The training example: embedding, norms and MLPs with 8-bit activations, the tied head's loss and all gradients in
one step.  The ends are exact to their operators' tolerances given what reaches them; the whole chain's gradients are
held to what its FP8 roundings can move them."""
import importlib.util
import os

import pytest
import torch

import fp8_fine_grained_x128_gb300 as fg

pytestmark = pytest.mark.gpu

spec = importlib.util.spec_from_file_location(
    "train_lm", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_lm.py"))
lm = importlib.util.module_from_spec(spec)
spec.loader.exec_module(lm)


def off(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def reference(model, ids, target):
    """The same model in 64 bits without any rounding: loss and gradients."""
    def leaf(t):
        return t.detach().double().requires_grad_()

    table = leaf(model.table.bf16)
    mats = [(leaf(b.up.bf16), leaf(b.down.bf16), leaf(b.norm.w)) for b in model.blocks]
    last = leaf(model.norm.w)

    def norm(x, w):
        return x * (x.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w

    here = (ids >= 0)[:, None]
    x = torch.where(here, table[ids.clamp(min=0).long()] * model.dim ** 0.5, 0.0)
    for up, down, w in mats:
        g, u = (norm(x, w) @ up.T).chunk(2, 1)
        x = x + (torch.nn.functional.silu(g) * u) @ down.T
    z = norm(x, last) @ table.T
    counts = target >= 0
    loss = torch.where(counts, torch.logsumexp(z, 1) - z.gather(1, target.clamp(min=0).long()[:, None])[:, 0], 0.0)
    (loss.sum() / counts.sum()).backward()
    return loss.detach(), table.grad, mats, last.grad


def test_step():
    V, D, F, T = 1000, 256, 384, 384
    model = lm.Model(V, D, F, blocks=2, seed=4)
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    target = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    target[::7] = -1
    ids[-40:], target[-40:] = -1, -100      # a padded batch
    loss = model.forward(ids, target).clone()
    model.backward()
    assert fg.device_status() == fg.OK
    counts = target >= 0
    assert not loss[~counts].any()

    # the ends, from what reaches them
    here = (ids >= 0)[:, None]
    assert torch.equal(model.x0, torch.where(here, model.table.bf16[ids.clamp(min=0).long()].float() * D ** 0.5, 0.0).bfloat16())
    z = model.y.double() @ model.table.bf16.double().T
    want = torch.where(counts, torch.logsumexp(z, 1) - z.gather(1, target.clamp(min=0).long()[:, None])[:, 0], 0.0)
    # D / 16 + 16 roundings of 2^-23 of a logit's terms, and those of a sum of V exponentials
    size = float((model.y.double().abs() @ model.table.bf16.double().abs().T).max())
    assert float((loss - want).abs().max()) <= 2 * ((D / 16 + 16) * 2.0 ** -23 * size + (V / 32 + 60) * 2.0 ** -23)

    # the chain: an E4M3 rounding moves an operand by at most 2^-4 of its norm; between a weight and the loss lie, on the
    # way there and back, the two operands of each product and what the norm and SwiGLU keep: at most 4 a product of 4
    ref_loss, ref_table, mats, ref_last = reference(model, ids, target)
    most = (1 + 2.0 ** -4) ** 16 - 1
    assert float((loss.sum() - ref_loss.sum()).abs() / ref_loss.sum()) <= 2.0 ** -4
    assert off(model.table.grad, ref_table) <= most / 4     # mostly the head's own product, which no FP8 reaches
    assert off(model.norm.grad, ref_last) <= most
    for b, (up, down, w) in zip(model.blocks, mats):
        assert off(b.up.grad, up.grad) <= most and off(b.down.grad, down.grad) <= most and off(b.norm.grad, w.grad) <= most
        # and they point the same way
        for mine, ref in ((b.up.grad, up.grad), (b.down.grad, down.grad)):
            assert float((mine.double() * ref).sum()) >= 0.9 * float(mine.double().norm() * ref.norm())

    # the same step again gives the same gradients, bit for bit
    first = [model.table.grad.clone(), model.norm.grad.clone(), model.blocks[0].up.grad.clone()]
    model.forward(ids, target)
    model.backward()
    assert all(torch.equal(a, b) for a, b in zip(first, (model.table.grad, model.norm.grad, model.blocks[0].up.grad)))
    model.update(1e-3, 1)
    assert fg.device_status() == fg.OK and bool(torch.isfinite(model.table.master).all())


def test_runs():
    lm.main(steps=2)
