"""fp8_paged_attention against a plain 64-bit attention, element by element
within bounds derived from the formats, over cache formats, head layouts,
group sizes, page sizes and lengths where it can go wrong."""
import pytest
import torch

import fp8_fine_grained_x128_gb300 as fg
from gpu_helpers import assert_status_ok, guarded
from paged_cases import Case

pytestmark = pytest.mark.gpu

SENTINEL = 123.0


@pytest.fixture(scope="module")
def workspace():
    return fg.new_attention_workspace()


def attend(c, ws, scale=None, stream=None):
    H = c.heads * c.group
    out, lse = guarded((c.tokens, H, c.dim), torch.bfloat16), guarded((c.tokens, H), torch.float32)
    out.fill_(SENTINEL)
    lse.fill_(SENTINEL)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    fg.paged_attention(c.cache(), c.batch(), c.q, out, ws, lse=lse, scale=scale, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    return out, lse


def check(c, out, lse, scale=None):
    assert_status_ok()
    ref, rlse, tol, ltol = c.reference(scale)
    own = ~torch.isnan(rlse[:, 0])
    assert bool((out[~own] == SENTINEL).all()) and bool((lse[~own] == SENTINEL).all()), "a row of no sequence written"
    got, want = out[own].double(), ref[own]
    assert bool(torch.isfinite(got).all())
    bad = (got - want).abs() > tol[own]
    assert not bool(bad.any()), (int(bad.sum()), float(((got - want).abs() / tol[own].clamp(min=1e-300)).max()))
    empty = torch.isinf(rlse[own])
    assert torch.equal(lse[own][empty].double(), rlse[own][empty])
    bad = (lse[own].double() - rlse[own]).abs()[~empty] > ltol[own][~empty]
    assert not bool(bad.any())


SINGLE = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 127), (1, 128), (1, 129), (1, 513), (1, 1000)]
CHUNKS = [(3, 3), (1, 70), (40, 40), (33, 161), (0, 50), (65, 300), (129, 129), (1, 1), (200, 457), (0, 0)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens", [SINGLE, CHUNKS], ids=["single", "chunks"])
def test_formats_and_lengths(workspace, kind, dim, lens):
    c = Case(lens, kind, dim=dim, seed=dim)
    check(c, *attend(c, workspace))


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 16, 17, 32])
@pytest.mark.parametrize("lens", [[(1, 77), (1, 300)], [(1, 40), (2, 130), (5, 260), (23, 150)]], ids=["single", "chunks"])
def test_group_sizes(workspace, group, lens):
    c = Case(lens, "bf16", heads=2, group=group, page=32, seed=group)
    check(c, *attend(c, workspace))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_page_sizes(workspace, page, kind):
    for seed, lens in enumerate(([(1, 700), (1, 255), (1, 257)], [(90, 700), (17, 255), (300, 513)])):
        c = Case(lens, kind, heads=3, group=2, page=page, seed=page + seed)
        check(c, *attend(c, workspace))


@pytest.mark.parametrize("layout", ["nhd", "padded", "joint"])
@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("e4m3", 64)])
def test_strides(workspace, layout, kind, dim):
    for lens in ([(1, 333), (1, 64)], [(70, 333), (9, 64)]):
        c = Case(lens, kind, dim=dim, layout=layout, page=32)
        check(c, *attend(c, workspace))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_rows_that_see_no_key(workspace, kind):
    """More new tokens than the cache counts: the first ones stand before position 0."""
    for lens in ([(1, 0), (1, 5), (2, 1), (4, 0)], [(40, 0), (40, 5), (200, 60), (150, 149)]):
        c = Case(lens, kind, seed=3)
        out, lse = attend(c, workspace)
        check(c, out, lse)


@pytest.mark.parametrize("lens", [[(1, 30), (1, 9)], [(30, 50), (7, 99)]], ids=["single", "chunks"])
def test_rows_of_no_sequence_are_left_alone(workspace, lens):
    c = Case(lens, "bf16", first=5, spare_tokens=9)
    c.q[:5] = float("nan")
    c.q[-9:] = float("nan")
    check(c, *attend(c, workspace))


@pytest.mark.parametrize("stale", [float("inf"), float("-inf"), float("nan"), -3.38e38])
def test_what_no_sequence_holds_is_not_read(workspace, stale):
    for lens in ([(1, 18), (1, 130)], [(50, 70), (140, 141)]):
        c = Case(lens, "bf16", stale=stale, page=64)
        check(c, *attend(c, workspace))


def test_long_caches_are_split(workspace):
    for kind, lens in (("bf16", [(1, 20011)]), ("e4m3", [(1, 30000), (1, 3)]), ("bf16", [(40, 9001)]),
                       ("e4m3", [(70, 9001), (1, 12)])):
        c = Case(lens, kind, heads=1, page=64, seed=9)
        check(c, *attend(c, workspace))


def test_many_sequences(workspace):
    lens = [(1, 1 + (37 * i) % 211) for i in range(300)]
    c = Case(lens, "bf16", heads=1, group=2, dim=64, seed=4)
    check(c, *attend(c, workspace))
    lens = [((5 * i) % 23, (5 * i) % 23 + (37 * i) % 90) for i in range(70)]
    c = Case(lens, "e4m3", heads=1, group=2, dim=64, seed=5)
    check(c, *attend(c, workspace))


DRAFTS = [(5, 700), (8, 8), (0, 40), (8, 3), (1, 1), (6, 129), (3, 9001), (7, 64), (8, 511), (2, 33), (4, 1000), (5, 6)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [1, 8], ids=["few pairs", "many pairs"])
def test_drafts(workspace, kind, dim, heads):
    """Up to 32 rows a sequence, among them none that sees a key, and one long cache: the batch's pairs
    decide which kernel takes them."""
    c = Case(DRAFTS, kind, heads=heads, dim=dim, page=32, seed=dim + heads)
    check(c, *attend(c, workspace))


@pytest.mark.parametrize("new", [8, 9, 16, 17])
def test_rows_around_the_choice_of_kernel(workspace, new):
    """Groups of 2 and 4 query heads: 16 to 68 rows."""
    for group in (2, 4):
        for kind in ("bf16", "e4m3"):
            c = Case([(new, 300 + 41 * i) for i in range(10)], kind, heads=5, group=group, seed=new + group)
            check(c, *attend(c, workspace))


def test_large_scores_and_scale(workspace):
    """Scores of hundreds: the softmax is one key nearly everywhere."""
    for lens in ([(1, 400)], [(60, 400)]):
        c = Case(lens, "bf16", q_std=60.0, seed=6)
        check(c, *attend(c, workspace))
        c = Case(lens, "e4m3", seed=7)
        check(c, *attend(c, workspace, scale=1e-4), scale=1e-4)


def test_growing_maximum(workspace):
    """Keys aligned with the query ever more strongly: the running maximum grows at every tile."""
    for new in (1, 80):
        c = Case([(new, 1500)], "bf16", heads=1, group=4, page=64, seed=8)
        ramp = torch.linspace(0.0, 6.0, 1500, device="cuda")
        one = torch.randn(128, device="cuda").bfloat16()
        c.q[:] = one
        j = torch.arange(1500, device="cuda")
        c.k[c.table[0, j // 64].long(), 0, j % 64] = (ramp[:, None] * one.float()).bfloat16()
        check(c, *attend(c, workspace))


def test_query_rows_as_column_range(workspace):
    for lens in ([(1, 50), (1, 8)], [(30, 50), (17, 80)]):
        c = Case(lens, "bf16")
        wide = torch.zeros((c.tokens, 24, 128), dtype=torch.bfloat16, device="cuda")
        wide[:, 2:10] = c.q
        c.q = wide[:, 2:10]
        check(c, *attend(c, workspace))


@pytest.mark.parametrize("lens", [[(1, 5000), (1, 77)], [(100, 5000), (1, 77)]], ids=["single", "chunks"])
def test_repeats_bit_for_bit_and_on_another_stream(workspace, lens):
    c = Case(lens, "e4m3", page=64)
    out, lse = attend(c, workspace)
    s = torch.cuda.Stream()
    for stream in (None, s):
        again, lse2 = attend(c, workspace, stream=stream)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert_status_ok()


def test_graph_replays_with_new_lengths(workspace):
    """The lengths and the page table are read on the device: one captured call serves every step."""
    c = Case([(1, 900), (1, 300)], "bf16", page=64)
    cache, batch = c.cache(), c.batch()
    out = torch.zeros_like(c.q)
    lse = torch.zeros(c.q.shape[:2], device="cuda")
    fg.paged_attention(cache, batch, c.q, out, workspace, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fg.paged_attention(cache, batch, c.q, out, workspace, lse=lse)
    for lens in ([(1, 900), (1, 300)], [(1, 17), (1, 299)], [(1, 1), (1, 128)]):
        c.lens = lens
        c.kv_lens.copy_(torch.tensor([kv for _, kv in lens], dtype=torch.int32))
        graph.replay()
        check(c, out, lse)


def test_offsets_past_32_bits(workspace):
    """A pool of more than 2^32 elements whose last pages are in use."""
    page, dim, pool = 64, 128, (1 << 32) // (64 * 128) + 40
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    c = Case([(1, 300), (20, 130)], "e4m3", heads=1, page=page)
    big_k = torch.zeros((pool, 1, page, dim), dtype=torch.uint8, device="cuda")
    big_v = torch.zeros((pool, 1, page, dim), dtype=torch.uint8, device="cuda")
    n = c.k.shape[0]
    big_k[-n:] = c.k.view(torch.uint8)
    big_v[-n:] = c.v.view(torch.uint8)
    want = attend(c, workspace)
    small = c.table.clone()
    c.table = torch.where(small >= 0, small + (pool - n), small)
    cache, batch = fg.PagedKV(big_k, big_v, c.k_scale, c.v_scale), c.batch()
    out, lse = torch.empty_like(c.q), torch.empty_like(want[1])
    fg.paged_attention(cache, batch, c.q, out, workspace, lse=lse)
    assert_status_ok()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("lens", [[(1, 100), (1, 40)], [(40, 100), (30, 40)]], ids=["single", "chunks"])
def test_bad_values_on_the_device_are_reported(workspace, lens):
    def status(c):
        attend(c, workspace)
        return fg.device_status()

    c = Case(lens, "bf16")
    c.table[0, 2] = c.k.shape[0]
    assert status(c) == fg.ERR_INVALID_ARG
    c = Case(lens, "e4m3")
    c.table[0, 2] = -1
    assert status(c) == fg.ERR_INVALID_ARG
    c = Case(lens, "bf16")
    c.kv_lens[1] = c.table.shape[1] * 16 + 1
    assert status(c) == fg.ERR_INVALID_ARG
    c = Case(lens, "bf16")
    c.kv_lens[1] = -1
    assert status(c) == fg.ERR_INVALID_ARG
    c = Case(lens, "bf16")
    check(c, *attend(c, workspace))   # the workspace is clean again


def test_empty_calls_write_nothing(workspace):
    c = Case([(1, 20)], "bf16")
    cache = c.cache()
    e = torch.empty((0, 8, 128), dtype=torch.bfloat16, device="cuda")
    fg.paged_attention(cache, c.batch(), e, e, workspace)
    none = fg.PagedBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                         torch.zeros((0, 1), dtype=torch.int32, device="cuda"), 0)
    out = torch.full_like(c.q, SENTINEL)
    fg.paged_attention(cache, none, c.q, out, workspace)
    assert_status_ok()
    assert bool((out == SENTINEL).all())


def test_refusals(workspace):
    c = Case([(1, 20)], "bf16")
    cache, batch, out = c.cache(), c.batch(), torch.empty_like(c.q)
    with pytest.raises(TypeError, match="PagedKV"):
        fg.paged_attention(c.k, batch, c.q, out, workspace)
    with pytest.raises(TypeError, match="dtype"):
        fg.paged_attention(cache, batch, c.q.float(), out, workspace)
    with pytest.raises(ValueError, match="expected"):
        fg.paged_attention(cache, batch, c.q, out[:, :4], workspace)
    with pytest.raises(ValueError, match="contiguous"):
        fg.paged_attention(cache, batch, c.q.transpose(0, 1).contiguous().transpose(0, 1)[:, ::2],
                           out[:, :4].contiguous(), workspace)
    with pytest.raises(ValueError, match="needs"):
        fg.paged_attention(cache, batch, c.q, out, workspace[:8])
    with pytest.raises(ValueError, match="needs"):
        fg.paged_attention(cache, batch, c.q, out, workspace, lse=torch.empty(3, device="cuda"))
    with pytest.raises(fg.Fp8Error) as e:   # 8 query heads over 3 cache heads
        fg.paged_attention(fg.PagedKV(c.k[:, [0, 1, 0]], c.v[:, [0, 1, 0]]), batch, c.q, out, workspace)
    assert e.value.code == fg.ERR_INVALID_ARG
    with pytest.raises(fg.Fp8Error) as e:
        fg.paged_attention(cache, batch, c.q, out, workspace, scale=float("nan"))
    assert e.value.code == fg.ERR_INVALID_ARG
    k = torch.zeros((2, 2, 24, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fg.Fp8Error) as e:
        fg.paged_attention(fg.PagedKV(k, k), batch, c.q, out, workspace)
    assert e.value.code == fg.ERR_UNSUPPORTED
    k = torch.zeros((2, 2, 16, 136), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((1, 8, 96), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fg.Fp8Error) as e:
        fg.paged_attention(fg.PagedKV(k[..., :96], k[..., :96]), batch, q, q.clone(), workspace)
    assert e.value.code == fg.ERR_UNSUPPORTED
    k = torch.zeros((2, 2, 16, 132), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fg.Fp8Error) as e:
        fg.paged_attention(fg.PagedKV(k[..., :128], k[..., :128]), batch, c.q, out, workspace)
    assert e.value.code == fg.ERR_ALIGNMENT
    with pytest.raises(ValueError, match="no scales"):
        fg.PagedKV(c.k, c.v, torch.ones(1, device="cuda"))
    with pytest.raises(ValueError, match="like k"):
        fg.PagedKV(c.k, c.v[:, :1])
    with pytest.raises(TypeError, match="dtype"):
        fg.PagedBatch(c.q_offsets.long(), c.kv_lens, c.table, 1)
    with pytest.raises(ValueError, match="needs"):
        fg.PagedBatch(c.q_offsets, c.kv_lens[:0], c.table, 1)
    assert_status_ok()
