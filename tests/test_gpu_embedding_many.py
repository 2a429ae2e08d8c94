"""The embedding's gradient over millions of tokens, and on a stream of its own."""
import pytest
import torch

import fp8_fine_grained_x128_gb300 as fg

pytestmark = pytest.mark.gpu


def case(T, V, D, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(-1, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    return ids, torch.randint(-2, 3, (T, D), generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("T,V", [(65537, 100), (1 << 20, 600), (3000001, 300000), (1 << 22, 1)])
def test_whole_numbers_are_exact(T, V):
    """Small whole numbers, fewer than 2^24 of them in absolute sum: every sum is exact in FP32."""
    D = 16
    ids, dout = case(T, V, D)
    dw = torch.full((V, D), 3.0, device="cuda")
    fg.embedding_bwd(ids, dout, dw, fg.new_embedding_workspace(T, V, D))
    here = ids >= 0
    want = torch.zeros((V, D), dtype=torch.float64, device="cuda").index_add_(0, ids[here].long(), dout[here].double())
    assert torch.equal(dw.double(), want) and fg.device_status() == fg.OK


def test_time_grows_with_the_tokens():
    """16 times the tokens take no more than twice 16 times as long (work that grew with the square took 256 times)."""
    V, D = 50000, 8

    def shortest(T):
        ids, dout = case(T, V, D)
        dw, ws = torch.empty((V, D), device="cuda"), fg.new_embedding_workspace(T, V, D)
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            fg.embedding_bwd(ids, dout, dw, ws)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times[1:])

    assert shortest(1 << 24) <= 32 * shortest(1 << 20)


@pytest.mark.parametrize("T", [500, 5000, 70000])
def test_on_another_stream(T):
    V, D = 2000, 64
    ids, dout = case(T, V, D, 1)

    def step():
        dw, out = torch.ones((V, D), device="cuda"), torch.empty_like(dout)
        fg.embedding_bwd(ids, dout, dw, fg.new_embedding_workspace(T, V, D), accumulate=True)
        fg.embedding_fwd(ids, dw.bfloat16(), out, scale=0.5)
        return dw, out

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(1000000)
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and fg.device_status() == fg.OK
