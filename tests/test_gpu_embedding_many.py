"""The embedding's gradient over millions of tokens."""
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
