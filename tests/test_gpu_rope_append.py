"""fp8_rope_append_kv: the rotation within bounds derived from FP32 and the
output formats, unrotated values bit for bit against the oracle's encoder,
every untouched cache row unchanged, and the device-side refusals."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_x128_gb300 as fg
import oracle
from gpu_helpers import assert_status_ok, guarded
from paged_cases import FMAX, Case

pytestmark = pytest.mark.gpu

LENS = [(1, 1), (3, 40), (0, 9), (17, 17), (1, 200), (33, 64)]


def inputs(c, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H = c.heads * c.group
    wide = torch.randn((c.tokens, (H + 2 * c.heads) * c.dim), generator=g, device="cuda").bfloat16()
    parts = wide.split([H * c.dim, c.heads * c.dim, c.heads * c.dim], 1)
    return [p.unflatten(1, (-1, c.dim)) for p in parts]


def table(n, rot):
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
        -torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotated(x, rope, pos, interleaved):
    """The pairs turned in 64 bits, and the sum of the absolute products."""
    x = x.double()
    rot = rope.shape[1]
    c, s = rope[pos, :rot // 2].double()[:, None], rope[pos, rot // 2:].double()[:, None]
    out, mag = x.clone(), x.abs()
    if interleaved:
        ia, ib = slice(0, rot, 2), slice(1, rot, 2)
    else:
        ia, ib = slice(0, rot // 2), slice(rot // 2, rot)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia], mag[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return out, mag


def places(c):
    """(token, sequence, position) of every token of a sequence."""
    rows, at = [], c.first
    for b, (n, kv) in enumerate(c.lens):
        rows += [(at + i, b, kv - n + i) for i in range(n)]
        at += n
    return [torch.tensor(v, device="cuda") for v in zip(*rows)]


def ulp_tol(ref, mag, kind):
    """Half an ulp of the format at the reference, plus three FP32 roundings of the products."""
    bits, emin = {"bf16": (8, -126), "e4m3": (4, -6), "e5m2": (3, -14)}[kind]
    e = torch.floor(torch.log2(ref.abs().clamp(min=2.0 ** emin)))
    return 2.0 ** (e - bits) * 1.0001 + mag * 3 * 2.0 ** -24


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind,dim,rot,layout,page", [
    ("bf16", 128, 128, "hnd", 16), ("bf16", 64, 32, "nhd", 32), ("e4m3", 128, 128, "padded", 64),
    ("e4m3", 64, 64, "joint", 128), ("e5m2", 128, 48, "nhd", 256), ("bf16", 128, 16, "joint", 16), ("e5m2", 64, 64, "hnd", 16)])
def test_append(kind, dim, rot, layout, page, interleaved):
    c = Case(LENS, kind, heads=3, group=3, dim=dim, page=page, layout=layout, seed=rot, first=2, spare_tokens=4, stale=None)
    q, k, v = inputs(c)
    rope = table(211, rot)
    q_out = guarded(tuple(q.shape), torch.bfloat16)
    q_out.fill_(77.0)
    before = c.k.float(), c.v.float()
    fg.rope_append_kv(c.cache(), c.batch(), k, v, rope, q=q, q_out=q_out, interleaved=interleaved)
    assert_status_ok()
    tok, seq, pos = places(c)
    mine = torch.zeros(c.tokens, dtype=torch.bool, device="cuda")
    mine[tok] = True
    assert bool((q_out[~mine] == 77.0).all())
    ref, mag = rotated(q[tok], rope, pos, interleaved)
    assert bool(((q_out[tok].double() - ref).abs() <= ulp_tol(ref, mag, "bf16")).all())
    pg, r = c.table[seq, pos // page].long(), pos % page
    ref, mag = rotated(k[tok], rope, pos, interleaved)
    if kind != "bf16":
        ref, mag = ref / c.k_scale.double(), mag / c.k_scale.double()
        ref = ref.clamp(-FMAX[kind], FMAX[kind])
    got = c.k.float()[pg, :, r].double()
    assert bool(((got - ref).abs() <= ulp_tol(ref, mag, kind)).all())
    # values (and the keys' unrotated elements) exactly
    want_v = v[tok]
    if kind == "bf16":
        assert torch.equal(c.v[pg, :, r], want_v)
        assert torch.equal(c.k[pg, :, r][..., rot:], k[tok][..., rot:])
    else:
        fmt = {"e4m3": oracle.E4M3, "e5m2": oracle.E5M2}[kind]
        for pages, src, s, lo in ((c.v, want_v, c.v_scale, 0), (c.k, k[tok], c.k_scale, rot)):
            x = src[..., lo:].float().cpu().numpy() / s.cpu().numpy()
            codes = pages.view(torch.uint8)[pg, :, r][..., lo:].cpu().numpy()
            assert np.array_equal(codes, oracle.fp8_encode(x.astype(np.float32), fmt).reshape(codes.shape))
    # nothing else moved
    touched = torch.zeros((c.k.shape[0], page), dtype=torch.bool, device="cuda")
    touched[pg, r] = True
    for pages, old in ((c.k, before[0]), (c.v, before[1])):
        assert torch.equal(pages.float().transpose(1, 2)[~touched], old.transpose(1, 2)[~touched])


def test_in_place_queries_and_keys_alone():
    c = Case(LENS, "bf16")
    q, k, v = inputs(c)
    rope = table(211, 128)
    out = torch.empty(tuple(q.shape), dtype=torch.bfloat16, device="cuda")
    fg.rope_append_kv(c.cache(), c.batch(), k, v, rope, q=q, q_out=out)
    first = c.k.clone(), c.v.clone()
    fg.rope_append_kv(c.cache(), c.batch(), k, v, rope, q=q, q_out=q)
    assert torch.equal(q, out)
    c.k.zero_()
    c.v.zero_()
    fg.rope_append_kv(c.cache(), c.batch(), k, v, rope)
    tok, seq, pos = places(c)
    pg, r = c.table[seq, pos // c.page].long(), pos % c.page
    for pages, old in ((c.k, first[0]), (c.v, first[1])):
        assert torch.equal(pages[pg, :, r], old[pg, :, r])
    assert_status_ok()


def test_no_rotation():
    c = Case(LENS, "bf16")
    q, k, v = inputs(c)
    out = torch.empty(tuple(q.shape), dtype=torch.bfloat16, device="cuda")
    fg.rope_append_kv(c.cache(), c.batch(), k, v, q=q, q_out=out)
    assert torch.equal(out, q)
    tok, seq, pos = places(c)
    pg, r = c.table[seq, pos // c.page].long(), pos % c.page
    assert torch.equal(c.k[pg, :, r], k[tok]) and torch.equal(c.v[pg, :, r], v[tok])
    assert_status_ok()


@pytest.mark.parametrize("scale", [1e-30, 1e-42, 3e38])
def test_extreme_scales_saturate_or_vanish(scale):
    """Scales outside the packed division's range and quotients past FP32."""
    for kind, fmt in (("e4m3", oracle.E4M3), ("e5m2", oracle.E5M2)):
        c = Case([(20, 20)], kind)
        c.v_scale = torch.tensor([scale], device="cuda")
        c.k_scale = torch.tensor([scale], device="cuda")
        q, k, v = inputs(c)
        fg.rope_append_kv(c.cache(), c.batch(), k, v)
        tok, seq, pos = places(c)
        pg, r = c.table[seq, pos // c.page].long(), pos % c.page
        with np.errstate(over="ignore"):
            x = v[tok].float().cpu().numpy() / np.float32(c.v_scale.item())
        codes = c.v.view(torch.uint8)[pg, :, r].cpu().numpy()
        assert np.array_equal(codes, oracle.fp8_encode(x.astype(np.float32), fmt).reshape(codes.shape))
        assert_status_ok()


def test_many_sequences_find_their_tokens():
    lens = [((7 * i) % 5, (7 * i) % 5 + (13 * i) % 60) for i in range(333)]
    c = Case(lens, "bf16", heads=1, group=1, dim=64)
    q, k, v = inputs(c)
    fg.rope_append_kv(c.cache(), c.batch(), k, v)
    tok, seq, pos = places(c)
    pg, r = c.table[seq, pos // c.page].long(), pos % c.page
    assert torch.equal(c.k[pg, :, r], k[tok]) and torch.equal(c.v[pg, :, r], v[tok])
    assert_status_ok()


def test_device_side_refusals():
    def status(change, rope=None, kind="bf16"):
        c = Case([(4, 30), (2, 9)], kind)
        q, k, v = inputs(c)
        change(c, k, v)
        fg.rope_append_kv(c.cache(), c.batch(), k, v, rope)
        return fg.device_status()

    assert status(lambda c, k, v: None) == fg.OK
    assert status(lambda c, k, v: c.table.__setitem__((0, 1), c.k.shape[0])) == fg.ERR_INVALID_ARG
    assert status(lambda c, k, v: c.table.__setitem__((1, 0), -1)) == fg.ERR_INVALID_ARG
    assert status(lambda c, k, v: c.kv_lens.__setitem__(0, 16 * c.table.shape[1] + 1)) == fg.ERR_INVALID_ARG
    assert status(lambda c, k, v: c.kv_lens.__setitem__(1, 1)) == fg.ERR_INVALID_ARG      # a token before position 0
    assert status(lambda c, k, v: None, table(29, 128)) == fg.ERR_INVALID_ARG             # the table ends at 28
    for kind in ("bf16", "e4m3"):
        for bad in (float("inf"), float("nan")):
            assert status(lambda c, k, v: k.__setitem__((3, 1, 5), bad), kind=kind) == fg.ERR_NONFINITE
            assert status(lambda c, k, v: v.__setitem__((5, 0, 127), bad), kind=kind) == fg.ERR_NONFINITE


def test_host_side_refusals():
    c = Case([(4, 30)], "bf16")
    q, k, v = inputs(c)
    cache, batch, rope = c.cache(), c.batch(), table(50, 128)
    with pytest.raises(ValueError, match="both or neither"):
        fg.rope_append_kv(cache, batch, k, v, rope, q=q)
    with pytest.raises(ValueError, match="expected"):
        fg.rope_append_kv(cache, batch, k[:, :1], v, rope)
    with pytest.raises(ValueError, match="expected"):
        fg.rope_append_kv(cache, batch, k, v[:2], rope)
    with pytest.raises(TypeError, match="dtype"):
        fg.rope_append_kv(cache, batch, k, v, rope.double())
    for r in (8, 24):
        with pytest.raises(fg.Fp8Error) as e:
            fg.rope_append_kv(cache, batch, k, v, rope[:, :r].contiguous())
        assert e.value.code == fg.ERR_SHAPE
    with pytest.raises(fg.Fp8Error) as e:
        fg.rope_append_kv(cache, batch, k, v, torch.zeros((50, 144), device="cuda"))
    assert e.value.code == fg.ERR_SHAPE
    odd = torch.zeros((4, 2 * 128 + 4), dtype=torch.bfloat16, device="cuda")[:, 4:].unflatten(1, (2, 128))
    with pytest.raises(fg.Fp8Error) as e:
        fg.rope_append_kv(cache, batch, odd, v, rope)
    assert e.value.code == fg.ERR_ALIGNMENT
    assert_status_ok()
