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
