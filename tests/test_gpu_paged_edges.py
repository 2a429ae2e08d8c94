"""The paged operators at the edges of their contract."""
import pytest
import torch

import fp8_fine_grained_x128_gb300 as fg
from gpu_helpers import assert_status_ok
from paged_cases import Case
from test_gpu_paged_attention import attend, check
from test_gpu_rope_append import inputs, places

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def workspace():
    return fg.new_attention_workspace()


# Changes that put a value of the batch's arrays out of its range, and the sequences that have to be refused
# (None: which tokens are whose is not defined).  The batch: tokens 0-3, 4-9 and 10-11.
LENS = [(4, 30), (6, 21), (2, 9)]
BAD = {
    "last offset past the tokens": (lambda c: c.q_offsets.__setitem__(3, c.tokens + 5), {2}),
    "offsets decrease": (lambda c: c.q_offsets.__setitem__(2, 2), None),
    "negative offset": (lambda c: c.q_offsets.__setitem__(0, -1), {0}),
    "more new tokens than max_new": (lambda c: setattr(c, "max_new", 5), {1}),
    "length past the page table": (lambda c: c.kv_lens.__setitem__(0, 16 * c.table.shape[1] + 1), {0}),
    "negative length": (lambda c: c.kv_lens.__setitem__(2, -3), {2}),
}


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_refuses_sequences_out_of_range(bad, kind):
    """Recorded, nothing of the refused sequences written, and no cached row of before in any case."""
    change, refused = BAD[bad]
    c = Case(LENS, kind, heads=1, group=1, spare_tokens=3, stale=None)
    q, k, v = inputs(c)
    tok, seq, pos = places(c)
    pg, r = c.table[seq, pos // c.page].long(), pos % c.page
    before = c.k.float(), c.v.float()
    fg.rope_append_kv(c.cache(), c.batch(), k, v)
    assert_status_ok()
    want = c.k.float(), c.v.float()
    for pages, old in zip((c.k, c.v), before):
        pages.copy_(old.to(pages.dtype))
    change(c)
    fg.rope_append_kv(c.cache(), c.batch(), k, v)
    assert fg.device_status() == fg.ERR_INVALID_ARG
    new = torch.zeros((c.k.shape[0], c.page), dtype=torch.bool, device="cuda")
    new[pg, r] = True
    for pages, old, full in zip((c.k, c.v), before, want):
        now = pages.float()
        assert torch.equal(now.transpose(1, 2)[~new], old.transpose(1, 2)[~new]), "a cached row of before overwritten"
        if refused is None:
            continue
        for b in range(len(LENS)):
            mine = seq == b
            rows = (old if b in refused else full)[pg[mine], :, r[mine]]
            assert torch.equal(now[pg[mine], :, r[mine]], rows), f"sequence {b}"


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("times", [1, 12], ids=["few rows", "many rows"])
def test_attention_refuses_sequences_out_of_range(workspace, bad, times):
    """Recorded, and the other sequences' outputs as they should be."""
    change, refused = BAD[bad]
    c = Case(LENS, "bf16", heads=1, group=times, spare_tokens=3)
    want, want_lse = attend(c, workspace)
    assert_status_ok()
    change(c)
    out, lse = attend(c, workspace)
    assert fg.device_status() == fg.ERR_INVALID_ARG
    if refused is not None:
        tok, seq, _ = places(c)
        for b in set(range(len(LENS))) - refused:
            assert torch.equal(out[tok[seq == b]], want[tok[seq == b]]) and torch.equal(lse[tok[seq == b]], want_lse[tok[seq == b]])
    c = Case(LENS, "bf16", heads=1, group=times)
    check(c, *attend(c, workspace))   # the workspace is clean again


def test_sequences_out_of_range_without_a_token(workspace):
    """Offsets past the tokens that no row falls to are recorded too; the length of a sequence without new
    tokens is nobody's business."""
    for offsets, lens, code in (([0, 4, 9], [30, 20], fg.ERR_INVALID_ARG), ([0, 4, 4], [30, -5], fg.OK),
                                ([0, 4] + [4] * 700 + [6], [30] + [0] * 701, fg.ERR_INVALID_ARG)):
        c = Case([(4, 30)], "bf16", heads=1, group=1)
        q, k, v = inputs(c)
        table = c.table.repeat(len(lens), 1)
        batch = fg.PagedBatch(torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                              torch.tensor(lens, dtype=torch.int32, device="cuda"), table, 5)
        fg.rope_append_kv(c.cache(), batch, k, v)
        assert fg.device_status() == code
        fg.paged_attention(c.cache(), batch, c.q, torch.empty_like(c.q), workspace)
        assert fg.device_status() == code


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("dim", [64, 128])
def test_many_units_of_one_or_two_tiles(workspace, kind, dim):
    """Every CTA goes from unit to unit all the time, with one half of rows or both."""
    lens = [(17 + i % 4 if i % 9 else 70, 70 + (37 * i) % 180) for i in range(220)]
    c = Case(lens, kind, heads=4, group=2, dim=dim, page=32, seed=dim)
    check(c, *attend(c, workspace))


KEYS, PAGE = 4500, 64
# sequences, new tokens of each, cache heads, query heads of a group: enough of them that a CTA's run holds a
# sequence's first and last keys
FORMS = {"few rows, one group": (100, 1, 8, 4), "few rows, two groups": (100, 5, 8, 4), "many rows": (80, 20, 4, 8)}


def shared_pages(workspace, kind, dim, form, columns, amps):
    """Sequences that share one sequence's pages, whose keys are `columns` [keys, n] in their first n elements
    and whose values are random; row r's query is amps[r] [n].  Scale 1.  Returns out, lse, and the 64-bit
    values: out, lse and the weighted mean of the absolute values."""
    seqs, new, heads, group = FORMS[form]
    g = torch.Generator(device="cuda").manual_seed(dim)
    pages = -(-KEYS // PAGE)
    dtype = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[kind]
    k = torch.zeros((pages * PAGE, heads, dim), device="cuda")
    k[:KEYS, :, :columns.shape[1]] = columns[:, None]
    v = torch.randn((pages * PAGE, heads, dim), generator=g, device="cuda")
    k, v = ((x.view(pages, PAGE, heads, dim).transpose(1, 2).contiguous()).to(dtype) for x in (k, v))
    tokens, H = seqs * new, heads * group
    q = torch.zeros((tokens, H, dim), dtype=torch.bfloat16, device="cuda")
    q[..., :columns.shape[1]] = amps[torch.arange(tokens * H, device="cuda") % amps.shape[0]].view(tokens, H, -1)
    ints = dict(dtype=torch.int32, device="cuda")
    batch = fg.PagedBatch(torch.arange(seqs + 1, **ints) * new, torch.full((seqs,), KEYS, **ints),
                          torch.arange(pages, **ints).repeat(seqs, 1), new)
    out, lse = torch.empty_like(q), torch.empty((tokens, H), device="cuda")
    fg.paged_attention(fg.PagedKV(k, v), batch, q, out, workspace, lse=lse, scale=1.0)
    assert_status_ok()
    kk, vv = (x.float().transpose(1, 2).reshape(-1, heads, dim)[:KEYS].double() for x in (k, v))
    after = torch.arange(KEYS, device="cuda") > (KEYS - new + torch.arange(tokens, device="cuda") % new)[:, None]
    ref, size, rlse = torch.empty(q.shape, dtype=torch.float64, device="cuda"), torch.empty_like(out, dtype=torch.float64), lse.double()
    for h in range(H):
        x = (q[:, h].double() @ kk[:, h // group].T).masked_fill(after, -float("inf"))
        w = torch.softmax(x, -1)
        ref[:, h], size[:, h], rlse[:, h] = w @ vv[:, h // group], w @ vv[:, h // group].abs(), torch.logsumexp(x, -1)
    return out.double(), lse.double(), ref, rlse, size


def half_ulp(ref):
    return 2.0 ** (torch.floor(torch.log2(ref.abs().clamp(min=2.0 ** -126))) - 8)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_one_late_key_carries_the_row(workspace, kind, dim, form):
    """A late key 2^5 to 2^8 times as heavy as the only other one that counts, the other one in the tile before
    its own and in the same 16 keys of it: too little for a lagging maximum to be raised.  The output is that
    key's value but for at most 2^-5 of the weight, so P's rounding must not show: 2^-13 of it from the light
    key in BF16, 2^-11 in FP16 (FP8 caches)."""
    at = 30 * 128 + 5
    c = torch.full((KEYS, 1), -16.0, device="cuda")
    c[at], c[at - 128] = 1.0, 0.0
    amps = (3.5 + torch.arange(128, device="cuda") / 64)[:, None]       # times log2 e: 5.05 to 7.91
    out, lse, ref, rlse, size = shared_pages(workspace, kind, dim, form, c, amps)
    bad = (out - ref).abs() > 2.0 ** -10 * size + half_ulp(ref)
    assert not bool(bad.any()), (int(bad.sum()), float(((out - ref).abs() / (2.0 ** -10 * size + half_ulp(ref))).max()))
    assert float((lse - rlse).abs().max()) < 2.0 ** -16


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("amp", [5.46875, 5.59375, 3.984375], ids=["steps of 7.89", "steps of 8.07", "steps of 5.75"])
def test_maximum_that_grows_from_tile_to_tile(workspace, kind, dim, form, amp):
    """Scores that rise in log2 by just under or just over 8 with every 128 keys, so that a lagging maximum is
    raised at every tile, every second, or after a part of one.  The weight lies on the last keys, evenly, and
    their rounding may go one way: P's unit roundoff, 2^-8 for BF16 and 2^-11 for FP16."""
    t = torch.arange(KEYS, device="cuda") // 128
    c = torch.stack([t % 8, t // 8], 1).float()      # exact in every format
    amps = torch.tensor([[amp, 8 * amp]], device="cuda")
    out, lse, ref, rlse, size = shared_pages(workspace, kind, dim, form, c, amps)
    # FP32: the score of up to 8 x 36 x amp rounds by 2^-24 of itself a few times, the sum of 128 keys by 2^-17
    e32 = 4 * 2.0 ** -24 * 36 * 8 * amp + 2.0 ** -16
    tol = (2.0 ** (-8 if kind == "bf16" else -11) + e32) * size + half_ulp(ref)
    bad = (out - ref).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), float(((out - ref).abs() / tol).max()))
    assert float((lse - rlse).abs().max()) < e32 + 2.0 ** -22 * float(rlse.abs().max())


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("lens", [[(1, 77), (1, 3)], [(5, 400), (1, 9)], [(1, 30000)], [(60, 300), (3, 3)], [(40, 9000)]],
                         ids=["single", "drafts", "long single", "chunks", "long chunk"])
def test_query_that_is_no_number_stays_in_its_row(workspace, kind, lens):
    """Output and LSE of that row are NaN (not the LSE of a row that sees no key); no other row changes."""
    c = Case(lens, kind, heads=1, page=64)
    want, want_lse = attend(c, workspace)
    c.q[0, 2, 17] = float("nan")
    out, lse = attend(c, workspace)
    assert_status_ok()
    assert bool(torch.isnan(out[0, 2]).all()) and bool(torch.isnan(lse[0, 2]))
    out[0, 2], lse[0, 2] = want[0, 2], want_lse[0, 2]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("lens", [[(1, 77), (1, 300)], [(5, 400), (8, 9)], [(60, 300), (3, 3)], [(40, 9000)]],
                         ids=["single", "drafts", "chunks", "long chunk"])
@pytest.mark.parametrize("signs", [(-1.0, 1.0), (1.0, -1.0), (-1.0, -1.0), (0.0, 1.0)], ids=str)
def test_scales_of_either_sign(workspace, kind, lens, signs):
    """An element stands for code times scale, whatever the scale's sign."""
    c = Case(lens, kind, heads=2, group=4, page=64)
    c.k_scale *= signs[0]
    c.v_scale *= signs[1]
    check(c, *attend(c, workspace))


@pytest.mark.parametrize("lens", [[(1, 77), (1, 300)], [(60, 300), (40, 90)]], ids=["single", "chunks"])
def test_scale_that_is_no_number_is_not_hidden(workspace, lens):
    for name in ("k_scale", "v_scale"):
        c = Case(lens, "e4m3", heads=2, group=4, page=64)
        setattr(c, name, torch.full((1,), float("nan"), device="cuda"))
        out, lse = attend(c, workspace)
        assert_status_ok()
        assert bool(torch.isnan(out).all())
        assert bool(torch.isnan(lse).all()) == (name == "k_scale")


def test_descriptors_do_not_go_stale(workspace):
    """An assigned max_new counts from the next call on; an assigned tensor, which the descriptor would not
    follow, is refused."""
    c = Case([(5, 60), (9, 30)], "e4m3")
    cache, batch = c.cache(), fg.PagedBatch(c.q_offsets, c.kv_lens, c.table, 1)
    out = torch.empty_like(c.q)
    fg.paged_attention(cache, batch, c.q, out, workspace)
    assert fg.device_status() == fg.ERR_INVALID_ARG
    batch.max_new = 9
    assert batch.max_new == 9
    fg.paged_attention(cache, batch, c.q, out, workspace)
    want, _ = attend(c, workspace)
    assert_status_ok()
    assert torch.equal(out, want)
    for n in (-1, 1 << 31):
        with pytest.raises(ValueError, match="max_new"):
            batch.max_new = n
    assert batch.max_new == 9
    for name in ("q_offsets", "kv_lens", "page_table"):
        with pytest.raises(AttributeError, match="marshalled"):
            setattr(batch, name, getattr(batch, name).clone())
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError, match="marshalled"):
            setattr(cache, name, getattr(cache, name).clone())


@pytest.mark.parametrize("group,new,past,dim", [(32, 264, 40, 64), (16, 529, 7, 128), (16, 1100, 300, 64), (8, 1024, 0, 64)],
                         ids=["33 units", "34 units", "69 units", "32 units"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_more_units_of_a_head_than_a_warp_has_lanes(workspace, kind, group, new, past, dim):
    """The walk counts 32 units of 256 rows a step; runs start inside later ones, and last units are short."""
    c = Case([(3, 50), (new, new + past), (20, 300)], kind, heads=2, group=group, dim=dim, page=64, seed=new)
    check(c, *attend(c, workspace))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("bound", [17, 40, 4096])
def test_max_new_above_every_sequence(workspace, kind, bound):
    """A captured step's bound: it alone chooses the kernels, the lengths on the device what they do."""
    for lens in ([(1, 1 + 67 * i) for i in range(30)], [(0, 5), (4, 4), (3, 700), (1, 2000), (0, 0)], [(0, 9), (0, 0)]):
        c = Case(lens, kind, heads=2, group=4, page=32, spare_tokens=2)
        c.max_new = bound
        check(c, *attend(c, workspace))


@pytest.mark.parametrize("seqs", [129, 700, 2500])
def test_batches_of_a_serving_size(workspace, seqs):
    """More sequences than a CTA has threads: single tokens alone, with a few chunks, and their append."""
    lens = [(1, 1 + (37 * i) % 90) for i in range(seqs)]
    for kind in ("bf16", "e4m3"):
        c = Case(lens, kind, heads=1, group=4, dim=64, seed=seqs)
        check(c, *attend(c, workspace))
        mixed = [(40, 300) if i % 401 == 128 else (1, 1 + (37 * i) % 90) if i % 3 else (0, i % 7) for i in range(seqs)]
        c = Case(mixed, kind, heads=1, group=4, dim=64, seed=seqs)
        check(c, *attend(c, workspace))
    c = Case(mixed, "bf16", heads=1, group=1, dim=64)
    q, k, v = inputs(c)
    fg.rope_append_kv(c.cache(), c.batch(), k, v)
    assert_status_ok()
    tok, seq, pos = places(c)
    pg, r = c.table[seq, pos // c.page].long(), pos % c.page
    assert torch.equal(c.k[pg, :, r], k[tok]) and torch.equal(c.v[pg, :, r], v[tok])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [[(1, 77), (1, 9000)], [(5, 400), (8, 9000)], [(60, 300), (40, 9000)]],
                         ids=["single", "drafts", "chunks"])
def test_outputs_without_lse(workspace, kind, lens):
    c = Case(lens, kind, heads=2, group=4, page=64)
    want, _ = attend(c, workspace)
    out = torch.empty_like(c.q)
    fg.paged_attention(c.cache(), c.batch(), c.q, out, workspace)
    assert_status_ok()
    assert torch.equal(out, want)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("lens", [[(1, 100), (1, 9000)], [(40, 100), (30, 9000)]], ids=["single", "chunks"])
def test_fp8_call_after_a_reported_page(workspace, kind, lens):
    """A page out of range in a sequence that is split over CTAs leaves nothing behind for the next call."""
    c = Case(lens, kind, heads=2, group=4, page=32)
    want, want_lse = attend(c, workspace)
    assert_status_ok()
    held = c.table[1, 100].clone()
    for bad in (c.k.shape[0], -1):
        c.table[1, 100] = bad
        out, lse = attend(c, workspace)
        assert fg.device_status() == fg.ERR_INVALID_ARG
        first = lens[0][0]
        assert torch.equal(out[:first], want[:first]) and torch.equal(lse[:first], want_lse[:first])
        c.table[1, 100] = held
        out, lse = attend(c, workspace)
        assert_status_ok()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
