"""The rollout example: projection, calibration, append and attention together,
prompts first and then captured single tokens, against 64-bit attention over what
the cache holds and against the projection's own keys and values."""
import importlib.util
import os

import pytest
import torch

import fp8_fine_grained_x128_gb300 as fg

pytestmark = pytest.mark.gpu

spec = importlib.util.spec_from_file_location(
    "paged_rollout", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_rollout.py"))
rollout = importlib.util.module_from_spec(spec)
spec.loader.exec_module(rollout)


def attention(layer, q, seq, length):
    """Attention of q [heads, dim] at position length - 1 of a sequence, in 64 bits over the cache."""
    j = torch.arange(length, device="cuda")
    page = layer.k.shape[2]
    pg = layer.table[seq, j // page].long()
    k = layer.k.float()[pg, :, j % page].double() * layer.k_scale.double()
    v = layer.v.float()[pg, :, j % page].double() * layer.v_scale.double()
    G = layer.Hq // layer.Hkv
    x = torch.einsum("hgd,jhd->hgj", q.double().view(layer.Hkv, G, -1), k) * layer.D ** -0.5
    return torch.einsum("hgj,jhd->hgd", torch.softmax(x, -1), v).reshape(layer.Hq, -1)


def close(got, want):
    """BF16 output and 16-bit probabilities: 2^-8 of the values' size, twice over."""
    assert float((got.double() - want).abs().max()) <= 2 * 2.0 ** -8 * float(want.abs().max().clamp(min=1.0))


def test_prompts_and_captured_steps():
    torch.manual_seed(3)
    lens = [200, 1, 77, 130]
    layer = rollout.Layer(hidden=512, q_heads=8, kv_heads=2, dim=128, page=32, seqs=4, max_len=256, seed=5)
    b = layer.buffers(sum(lens))
    b["x"][:sum(lens)].normal_()
    layer.prompts(b, lens)
    assert fg.device_status() == fg.OK
    start = 0
    for seq, n in enumerate(lens):
        close(b["out"][start + n - 1], attention(layer, b["q"][start + n - 1], seq, n))
        # the newest value row: the projection's, as the cache's format holds it
        pg, r = int(layer.table[seq, (n - 1) // 32]), (n - 1) % 32
        v = b["v"][start + n - 1].float()
        held = layer.v.float()[pg, :, r] * layer.v_scale
        assert bool(((held - v).abs() <= 2.0 ** -4 * v.abs() + 2.0 ** -10 * layer.v_scale).all())
        start += n
    one = layer.buffers(len(lens))
    graph = layer.capture_step(one)
    for step in range(1, 4):
        one["x"][:4].normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert fg.device_status() == fg.OK
        assert layer.kv_lens.tolist() == [n + step for n in lens]
        for seq, n in enumerate(lens):
            close(one["out"][seq], attention(layer, one["q"][seq], seq, n + step))
