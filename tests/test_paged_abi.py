"""Host-side argument validation of the paged cache entry points: bad calls
are refused with the documented status before anything is launched (no GPU)."""
import ctypes

import pytest

import fp8_fine_grained_x128_gb300 as fg
from fp8_fine_grained_x128_gb300 import build as fgbuild

GOOD, ODD = 4096, 4104   # never dereferenced; ODD is not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    fgbuild.build()
    return fg.lib()


def cache(**change):
    st = fg._PagedKV(GOOD, GOOD, 2 * 16 * 128, 16 * 128, 128, 2 * 16 * 128, 16 * 128, 128, None, None, fg.KV_BF16, 9, 16, 2, 128)
    for k, v in change.items():
        setattr(st, k, v)
    return ctypes.byref(st)


def batch(**change):
    st = fg._PagedBatch(GOOD, GOOD, GOOD, 4, 2, 4, 1)
    for k, v in change.items():
        setattr(st, k, v)
    return ctypes.byref(st)


BOTH = [
    (dict(k=None), {}, fg.ERR_INVALID_ARG), (dict(k=ODD), {}, fg.ERR_ALIGNMENT), (dict(v=ODD), {}, fg.ERR_ALIGNMENT),
    (dict(format=3), {}, fg.ERR_INVALID_ARG), (dict(k_scale=GOOD), {}, fg.ERR_INVALID_ARG),
    (dict(num_pages=0), {}, fg.ERR_INVALID_ARG), (dict(heads=0), {}, fg.ERR_INVALID_ARG),
    (dict(head_dim=96), {}, fg.ERR_UNSUPPORTED), (dict(page_size=24), {}, fg.ERR_UNSUPPORTED),
    (dict(page_size=8), {}, fg.ERR_UNSUPPORTED), (dict(page_size=512), {}, fg.ERR_UNSUPPORTED),
    (dict(k_row_stride=132), {}, fg.ERR_ALIGNMENT), (dict(v_page_stride=0), {}, fg.ERR_SHAPE),
    (dict(v_head_stride=-128), {}, fg.ERR_SHAPE), (dict(k_row_stride=64), {}, fg.ERR_SHAPE),
    (dict(k_page_stride=1 << 39), {}, fg.ERR_SHAPE),
    ({}, dict(seqs=-1), fg.ERR_INVALID_ARG), ({}, dict(seqs=65537), fg.ERR_INVALID_ARG),
    ({}, dict(max_new=-1), fg.ERR_INVALID_ARG), ({}, dict(page_table_ld=3), fg.ERR_SHAPE),
    ({}, dict(pages_per_seq=1 << 27, page_table_ld=1 << 27), fg.ERR_SHAPE), ({}, dict(page_table=None), fg.ERR_INVALID_ARG),
    ({}, dict(q_offsets=None), fg.ERR_INVALID_ARG), ({}, dict(kv_lens=None), fg.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("c,b,code", BOTH)
def test_cache_and_batch(lib, c, b, code):
    assert lib.fp8_paged_attention(cache(**c), batch(**b), 4, GOOD, 512, 4, 0.1, GOOD, 512, None, GOOD, None) == code
    assert lib.fp8_rope_append_kv(cache(**c), batch(**b), 4, GOOD, 512, 4, GOOD, 256, GOOD, 256, GOOD, 99, 128, 0, GOOD, 512,
                                  None) == code


def test_attention_operands(lib):
    def call(c=None, b=None, tokens=4, q=GOOD, ld=512, heads=4, scale=0.1, out=GOOD, out_ld=512, lse=None, ws=GOOD):
        return lib.fp8_paged_attention(c or cache(), b or batch(), tokens, q, ld, heads, scale, out, out_ld, lse, ws, None)

    assert lib.fp8_paged_attention(None, batch(), 4, GOOD, 512, 4, 0.1, GOOD, 512, None, GOOD, None) == fg.ERR_INVALID_ARG
    assert lib.fp8_paged_attention(cache(), None, 4, GOOD, 512, 4, 0.1, GOOD, 512, None, GOOD, None) == fg.ERR_INVALID_ARG
    assert call(tokens=-1) == fg.ERR_SHAPE
    assert call(tokens=1 << 30) == fg.ERR_SHAPE
    assert call(q=None) == fg.ERR_INVALID_ARG and call(q=ODD) == fg.ERR_ALIGNMENT
    assert call(ld=511) == fg.ERR_SHAPE and call(ld=516) == fg.ERR_ALIGNMENT
    assert call(heads=3) == fg.ERR_INVALID_ARG and call(heads=0) == fg.ERR_INVALID_ARG
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == fg.ERR_INVALID_ARG
    assert call(out=ODD) == fg.ERR_ALIGNMENT and call(out_ld=256) == fg.ERR_SHAPE
    assert call(lse=4098) == fg.ERR_ALIGNMENT
    assert call(ws=None) == fg.ERR_INVALID_ARG and call(ws=ODD) == fg.ERR_ALIGNMENT
    assert call(tokens=0) == fg.OK and call(b=batch(seqs=0)) == fg.OK


def test_append_operands(lib):
    def call(tokens=4, q=GOOD, q_ld=512, heads=4, k=GOOD, k_ld=256, v=GOOD, v_ld=256, rope=GOOD, n=99, rot=128, inter=0,
             out=GOOD, out_ld=512):
        return lib.fp8_rope_append_kv(cache(), batch(), tokens, q, q_ld, heads, k, k_ld, v, v_ld, rope, n, rot, inter, out,
                                      out_ld, None)

    assert call(q=None) == fg.ERR_INVALID_ARG and call(out=None) == fg.ERR_INVALID_ARG
    assert call(k=None) == fg.ERR_INVALID_ARG and call(v=ODD) == fg.ERR_ALIGNMENT
    assert call(k_ld=128) == fg.ERR_SHAPE and call(v_ld=260) == fg.ERR_ALIGNMENT
    assert call(rope=None) == fg.ERR_INVALID_ARG and call(rope=ODD) == fg.ERR_ALIGNMENT
    assert call(rot=120) == fg.ERR_SHAPE and call(rot=144) == fg.ERR_SHAPE and call(rot=-16) == fg.ERR_SHAPE
    assert call(n=-1) == fg.ERR_INVALID_ARG and call(inter=2) == fg.ERR_INVALID_ARG and call(heads=-1) == fg.ERR_INVALID_ARG
    assert call(tokens=0) == fg.OK


def test_workspace_is_refused_on_the_host():
    import torch
    with pytest.raises(ValueError, match="CUDA tensor"):
        fg.PagedKV(torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16), torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA tensor"):
        fg.PagedBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                      torch.zeros((1, 1), dtype=torch.int32), 1)
