"""Embedding lookup and its gradient against their definitions.  A sum of n rows in FP32, in any order, is off by at most
n 2^-24 of the rows' absolute sum (a rounding for each addition), the scale's product by 2^-24, a BF16 result by 2^-8."""
import math

import pytest
import torch

import fp8_fine_grained_x128_gb300 as fg

pytestmark = pytest.mark.gpu


def words(T, V, kind, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "one":
        ids = torch.full((T,), V - 1, device="cuda")
    elif kind == "few":
        ids = torch.randint(min(V, 3), (T,), generator=g, device="cuda")
    elif kind == "pad":
        ids = torch.randint(V, (T,), generator=g, device="cuda")
        ids[torch.rand(T, generator=g, device="cuda") < 0.5] = -1
    else:
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        ids = (float(V) ** u).long().clamp(max=V) - 1
    return ids.to(torch.int32)


SIZES = [(1, 1, 8), (1, 1000, 64), (31, 7, 16), (32, 600, 256), (33, 511, 264), (100, 512, 1000), (2048, 513, 128), (2049, 100003, 72),
         (5000, 262145, 64), (8192, 2000, 40), (8193, 700, 40), (9001, 32001, 520), (16385, 511, 24), (40000, 300000, 16), (65536, 1 << 18, 8),
         (65537, (1 << 18) - 1, 8), (150001, 3000, 16)]


@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("scale", [1.0, 0.37])
def test_forward(T, V, D, scale):
    ids = words(T, V, "pad", 1)
    wide = torch.randn((V, D + 8), device="cuda").bfloat16()
    w = wide[:, :D]
    out = torch.full((T + 1, D + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    fg.embedding_fwd(ids, w, out[:T, :D], scale=scale)
    assert fg.device_status() == fg.OK
    # one product of a BF16 and an FP32 value, rounded to FP32 and then to BF16, as torch's
    want = torch.where((ids >= 0)[:, None], w[ids.clamp(min=0).long()].float() * scale, 0.0).bfloat16()
    assert torch.equal(out[:T, :D], want)
    assert bool((out[T:] == 3).all()) and bool((out[:, D:] == 3).all())


@pytest.mark.parametrize("kind", ["zipf", "one", "few", "pad"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_gradient(T, V, D, kind):
    ids = words(T, V, kind, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    dout = torch.randn((T, D + 8), generator=g, device="cuda").bfloat16()[:, :D]
    here = ids >= 0
    at = ids[here].long()
    want = torch.zeros((V, D), dtype=torch.float64, device="cuda").index_add_(0, at, dout[here].double())
    size = torch.zeros((V, D), dtype=torch.float64, device="cuda").index_add_(0, at, dout[here].double().abs())
    n = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, at, torch.ones(at.numel(), dtype=torch.float64, device="cuda"))[:, None]
    scale = 1.3
    ws = fg.new_embedding_workspace(T, V, D)
    tol = (n + 2) * 2.0 ** -24 * size * scale
    for dtype, accumulate in ((torch.float32, False), (torch.float32, True), (torch.bfloat16, False)):
        wide = torch.full((V + 1, D + 8), 2.0, dtype=dtype, device="cuda")
        dw = wide[:V, :D]
        fg.embedding_bwd(ids, dout, dw, ws, scale=scale, accumulate=accumulate)
        assert fg.device_status() == fg.OK
        assert bool((wide[V:] == 2).all()) and bool((wide[:, D:] == 2).all())
        ref = want * torch.tensor(scale).float().double()
        t = tol
        if accumulate:
            ref, t = ref + 2.0, tol + 2.0 ** -24 * (ref + 2.0).abs() + tol * 2.0 ** -24
            assert bool((dw[(n == 0)[:, 0]] == 2).all())
        if dtype == torch.bfloat16:
            t = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
        assert bool(((dw.double() - ref).abs() <= t).all())
        again = torch.full_like(wide, 2.0)
        ws.fill_(255)       # any content of the workspace
        fg.embedding_bwd(ids, dout, again[:V, :D], ws, scale=scale, accumulate=accumulate)
        assert torch.equal(again, wide)


def test_whole_numbers_are_exact():
    """Small whole numbers: every sum is exact in FP32, whatever the pieces, so the result has to be equal."""
    T, V, D = 20000, 50, 320
    ids = words(T, V, "zipf", 4)
    dout = torch.randint(-8, 9, (T, D), device="cuda").bfloat16()
    dw = torch.empty((V, D), device="cuda")
    fg.embedding_bwd(ids, dout, dw, fg.new_embedding_workspace(T, V, D))
    want = torch.zeros((V, D), device="cuda", dtype=torch.float64).index_add_(0, ids.long(), dout.double())
    assert torch.equal(dw.double(), want)


def test_padding_holds_anything_and_bad_ids_are_recorded():
    T, V, D = 300, 40, 64
    ids = words(T, V, "pad", 5)
    dout = torch.randn((T, D), device="cuda").bfloat16()
    ws = fg.new_embedding_workspace(T, V, D)
    want = torch.empty((V, D), device="cuda")
    fg.embedding_bwd(ids, dout, want, ws)
    dout[ids < 0] = math.nan
    dw = torch.empty_like(want)
    fg.embedding_bwd(ids, dout, dw, ws)
    assert torch.equal(dw, want) and fg.device_status() == fg.OK
    bad = torch.where(ids < 0, torch.tensor(1 << 30, dtype=torch.int32, device="cuda"), ids)
    bad[ids < 0] += torch.arange(int((ids < 0).sum()), dtype=torch.int32, device="cuda")
    fg.embedding_bwd(bad, dout, dw, ws)
    assert torch.equal(dw, want) and fg.device_status() == fg.ERR_INVALID_ARG
    w, out = torch.randn((V, D), device="cuda").bfloat16(), torch.ones((T, D), device="cuda", dtype=torch.bfloat16)
    bad[0] = V
    fg.embedding_fwd(bad, w, out)
    assert fg.device_status() == fg.ERR_INVALID_ARG and bool((out[bad >= V] == 0).all())


@pytest.mark.parametrize("T", [300, 4000, 70000])
def test_captured(T):
    V, D = 3001, 128
    ids, dout = words(T, V, "zipf", 6), torch.randn((T, D), device="cuda").bfloat16()
    ws, dw = fg.new_embedding_workspace(T, V, D), torch.empty((V, D), device="cuda")
    fg.embedding_bwd(ids, dout, dw, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fg.embedding_bwd(ids, dout, dw, ws)
    ids.copy_(words(T, V, "few", 7))
    graph.replay()
    got = dw.clone()
    fg.embedding_bwd(ids, dout, dw, ws)
    assert torch.equal(got, dw) and fg.device_status() == fg.OK


def test_one_workspace_for_calls_of_many_sizes():
    ws = fg.new_embedding_workspace(70000, 5000, 1032)
    for T, V, D in ((70000, 5000, 8), (70000, 17, 1032), (1, 1, 1032), (3000, 5000, 512), (69999, 4999, 1024)):
        ids, dout = words(T, V, "zipf", 6), torch.randn((T, D), device="cuda").bfloat16()
        a, b = torch.empty((V, D), device="cuda"), torch.empty((V, D), device="cuda")
        fg.embedding_bwd(ids, dout, a, ws)
        fg.embedding_bwd(ids, dout, b, fg.new_embedding_workspace(T, V, D))
        assert torch.equal(a, b) and fg.device_status() == fg.OK


def test_no_tokens_or_words():
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    rows = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    dw = torch.ones((10, 64), device="cuda")
    ws = fg.new_embedding_workspace(0, 10, 64)
    fg.embedding_bwd(e, rows, dw, ws, accumulate=True)
    assert bool((dw == 1).all())
    fg.embedding_bwd(e, rows, dw, ws)
    assert not dw.any()
    fg.embedding_fwd(e, dw.bfloat16(), rows)
    out = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    fg.embedding_fwd(torch.full((2,), -1, dtype=torch.int32, device="cuda"), rows, out)     # nothing but padding, no words
    assert not out.any() and fg.device_status() == fg.OK


@pytest.mark.parametrize("T", [500, 5000, 70000])
def test_offsets_beyond_32_bits_full_size(T):
    """A table of more than 2^31 elements, ids at both ends and scattered."""
    V, D = 1100000, 2048
    g = torch.Generator(device="cuda").manual_seed(8)
    ids = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    ids[:4] = torch.tensor([V - 1, 0, V - 1, V - 2], dtype=torch.int32)
    w = torch.empty((V, D), dtype=torch.bfloat16, device="cuda")
    w.view(torch.int16).copy_((torch.arange(V, device="cuda") % 16384).to(torch.int16)[:, None].expand(V, D))
    out = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    fg.embedding_fwd(ids, w, out)
    assert torch.equal(out.view(torch.int16), (ids % 16384).to(torch.int16)[:, None].expand(T, D))
    del w
    dout = torch.randint(-4, 5, (T, D), generator=g, device="cuda").bfloat16()
    dw = torch.full((V, D), 3.0, device="cuda")
    fg.embedding_bwd(ids, dout, dw, fg.new_embedding_workspace(T, V, D))
    uniq, inv = torch.unique(ids, return_inverse=True)
    want = torch.zeros((uniq.numel(), D), device="cuda").index_add_(0, inv, dout.float())
    assert torch.equal(dw[uniq.long()], want)
    assert int((dw != 0).any(1).sum()) <= uniq.numel() and fg.device_status() == fg.OK
