"""Refusals of the embedding, norm, SwiGLU-checkpoint and cross-entropy entry points: the documented status before
anything touches the GPU (runs without one)."""
import ctypes
import random

import pytest
import torch

import fp8_fine_grained_x128_gb300 as fg
from fp8_fine_grained_x128_gb300 import build as fgbuild

P = 1 << 20            # a 16-byte aligned address that is never followed
S = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    fgbuild.build()
    return fg.lib()


def norm_fwd(lib, x=P, rows=4, cols=256, ldx=256, res=P, ldres=256, w=P, eps=1e-5, fmt=0, y=P, ldy=256, sum=P, ldsum=256, c=P, cs=P, rstd=P):
    return lib.fp8_rmsnorm_fwd_ckpt(x, rows, cols, ldx, res, ldres, w, eps, fmt, y, ldy, sum, ldsum, c, cs, rstd, S)


def norm_bwd(lib, c=P, cs=P, rstd=P, fmt=0, rows=4, cols=256, w=P, dy=P, lddy=256, dsum=P, lddsum=256, dx=P, lddx=256, dw=P, ws=P):
    return lib.fp8_rmsnorm_bwd_ckpt(c, cs, rstd, fmt, rows, cols, w, dy, lddy, dsum, lddsum, dx, lddx, dw, 0, ws, S)


@pytest.mark.parametrize("bad,status", [
    ({"cols": 250}, fg.ERR_SHAPE), ({"cols": 16512}, fg.ERR_SHAPE), ({"rows": -1}, fg.ERR_SHAPE), ({"rows": 1 << 31}, fg.ERR_SHAPE),
    ({"fmt": 2}, fg.ERR_INVALID_ARG), ({"eps": 0.0}, fg.ERR_INVALID_ARG), ({"eps": float("nan")}, fg.ERR_INVALID_ARG),
    ({"res": None}, fg.ERR_INVALID_ARG), ({"sum": None}, fg.ERR_INVALID_ARG), ({"x": None}, fg.ERR_INVALID_ARG),
    ({"rstd": None}, fg.ERR_INVALID_ARG), ({"x": P + 2}, fg.ERR_ALIGNMENT), ({"y": P + 8}, fg.ERR_ALIGNMENT), ({"c": P + 8}, fg.ERR_ALIGNMENT),
    ({"cs": P + 2}, fg.ERR_ALIGNMENT), ({"ldx": 260}, fg.ERR_ALIGNMENT), ({"ldy": 128}, fg.ERR_SHAPE), ({"ldsum": 128}, fg.ERR_SHAPE),
    ({"rows": 0, "x": None}, fg.OK)])
def test_norm_forward_refuses(lib, bad, status):
    assert norm_fwd(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [
    ({"cols": 100}, fg.ERR_SHAPE), ({"rows": -1}, fg.ERR_SHAPE), ({"fmt": -1}, fg.ERR_INVALID_ARG), ({"dw": None}, fg.ERR_INVALID_ARG),
    ({"dw": P + 2}, fg.ERR_ALIGNMENT), ({"ws": None}, fg.ERR_INVALID_ARG), ({"ws": P + 8}, fg.ERR_ALIGNMENT), ({"dy": None}, fg.ERR_INVALID_ARG),
    ({"dx": P + 4}, fg.ERR_ALIGNMENT), ({"lddx": 128}, fg.ERR_SHAPE), ({"dsum": P + 2}, fg.ERR_ALIGNMENT), ({"lddy": 257}, fg.ERR_ALIGNMENT),
    ({"cols": 0}, fg.OK)])
def test_norm_backward_refuses(lib, bad, status):
    assert norm_bwd(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [
    ({"F": 130}, fg.ERR_SHAPE), ({"rows": -1}, fg.ERR_SHAPE), ({"fmt": 5}, fg.ERR_INVALID_ARG), ({"a": None}, fg.ERR_INVALID_ARG),
    ({"o": P + 8}, fg.ERR_ALIGNMENT), ({"c": P + 4}, fg.ERR_ALIGNMENT), ({"cs": None}, fg.ERR_INVALID_ARG), ({"rows": 0, "a": None}, fg.OK)])
def test_swiglu_refuses(lib, bad, status):
    def fwd(a=P, rows=4, F=256, fmt=0, o=P, c=P, cs=P):
        return lib.fp8_swiglu_fwd_ckpt(a, rows, F, fmt, o, c, cs, S)

    def bwd(a=P, rows=4, F=256, fmt=0, o=P, c=P, cs=P):
        return lib.fp8_swiglu_bwd_ckpt(c, cs, a, rows, F, fmt, o, S)

    assert fwd(**bad) == status and bwd(**bad) == status


@pytest.mark.parametrize("bad,status", [
    ({"dim": 12}, fg.ERR_SHAPE), ({"T": -1}, fg.ERR_SHAPE), ({"T": (1 << 30) + 1}, fg.ERR_SHAPE), ({"V": (1 << 30) + 1}, fg.ERR_SHAPE),
    ({"scale": float("nan")}, fg.ERR_INVALID_ARG), ({"ids": None}, fg.ERR_INVALID_ARG), ({"ids": P + 2}, fg.ERR_ALIGNMENT),
    ({"rows": None}, fg.ERR_INVALID_ARG), ({"rows": P + 8}, fg.ERR_ALIGNMENT), ({"ld": 56}, fg.ERR_SHAPE), ({"ld": 68}, fg.ERR_ALIGNMENT),
    ({"dim": 0}, fg.OK)])
def test_embedding_refuses(lib, bad, status):
    def fwd(ids=P, T=4, V=10, dim=64, rows=P, ld=64, scale=1.0):
        return lib.fp8_embedding_fwd(ids, T, P, V, dim, 64, scale, rows, ld, S)

    def bwd(ids=P, T=4, V=10, dim=64, rows=P, ld=64, scale=1.0):
        return lib.fp8_embedding_bwd(ids, T, rows, ld, V, dim, scale, P, 0, 64, 0, P, S)

    assert fwd(**bad) == status and bwd(**bad) == status


def test_embedding_gradient_refuses(lib):
    def f(dw=P, dtype=0, ld=64, acc=0, ws=P):
        return lib.fp8_embedding_bwd(P, 4, P, 64, 10, 64, 1.0, dw, dtype, ld, acc, ws, S)

    assert f(acc=1) == fg.ERR_UNSUPPORTED                  # BF16 results are not added to
    assert f(dtype=2) == fg.ERR_INVALID_ARG
    assert f(dw=None) == fg.ERR_INVALID_ARG and f(dw=P + 8) == fg.ERR_ALIGNMENT
    assert f(ws=None) == fg.ERR_INVALID_ARG and f(ws=P + 4) == fg.ERR_ALIGNMENT
    assert f(ld=60) == fg.ERR_SHAPE and f(ld=68) == fg.ERR_ALIGNMENT


def xent(lib, back, x=P, T=4, D=64, ldx=64, w=P, V=10, ldw=64, t=P, scale=1.0, loss=P, lse=P, ws=P, dl=P, dz=P, dx=P, lddx=64, dw=P, dtype=0,
         lddw=64, acc=0):
    if not back:
        return lib.fp8_linear_xent_fwd(x, T, D, ldx, w, V, ldw, t, scale, loss, lse, ws, S)
    return lib.fp8_linear_xent_bwd(x, T, D, ldx, w, V, ldw, t, scale, loss, lse, dl, dz, dx, lddx, dw, dtype, lddw, acc, ws, S)


@pytest.mark.parametrize("bad,status", [
    ({"D": 63}, fg.ERR_SHAPE), ({"T": -1}, fg.ERR_SHAPE), ({"V": 0}, fg.ERR_SHAPE), ({"D": 0}, fg.ERR_SHAPE), ({"T": 1 << 28}, fg.ERR_SHAPE), ({"T": 1 << 24, "V": 1 << 22}, fg.ERR_SHAPE),
    ({"scale": 0.0}, fg.ERR_INVALID_ARG), ({"scale": -1.0}, fg.ERR_INVALID_ARG), ({"scale": float("inf")}, fg.ERR_INVALID_ARG),
    ({"x": None}, fg.ERR_INVALID_ARG), ({"w": P + 2}, fg.ERR_ALIGNMENT), ({"ldx": 56}, fg.ERR_SHAPE), ({"ldw": 65}, fg.ERR_ALIGNMENT),
    ({"t": None}, fg.ERR_INVALID_ARG), ({"t": P + 1}, fg.ERR_ALIGNMENT), ({"loss": None}, fg.ERR_INVALID_ARG), ({"lse": P + 2}, fg.ERR_ALIGNMENT),
    ({"ws": None}, fg.ERR_INVALID_ARG), ({"ws": P + 8}, fg.ERR_ALIGNMENT)])
def test_xent_refuses(lib, bad, status):
    assert xent(lib, False, **bad) == status and xent(lib, True, **bad) == status


def test_xent_gradient_refuses(lib):
    def f(**kw):
        return xent(lib, True, **kw)

    assert f(acc=1) == fg.ERR_UNSUPPORTED and f(dtype=3) == fg.ERR_INVALID_ARG
    assert f(dl=None) == fg.ERR_INVALID_ARG and f(dl=P + 2) == fg.ERR_ALIGNMENT and f(dz=P + 2) == fg.ERR_ALIGNMENT
    assert f(dx=None) == fg.ERR_INVALID_ARG and f(lddx=32) == fg.ERR_SHAPE and f(dw=P + 8) == fg.ERR_ALIGNMENT
    assert f(dtype=1, lddw=66) == fg.ERR_ALIGNMENT
    assert f(T=0, x=None, dtype=1, acc=1) == fg.OK         # nothing to add


def test_workspace_sizes(lib):
    assert lib.fp8_linear_xent_workspace_bytes(-1, 10, 64, 0) == 0 and lib.fp8_linear_xent_workspace_bytes(4, 10, 63, 1) == 0
    small = lib.fp8_linear_xent_workspace_bytes(8192, 128000, 4096, 0)
    assert 0 < small < 8192 * 128000 * 2 // 16              # far below the logits
    assert lib.fp8_linear_xent_workspace_bytes(8192, 128000, 4096, 1) < 8192 * 128000 * 2 // 4
    assert lib.fp8_embedding_workspace_bytes(100, 10, 12) == 0 and lib.fp8_rmsnorm_workspace_bytes(1 << 20) == 0


@pytest.mark.parametrize("bytes_of", [lambda L, *s: L.fp8_embedding_workspace_bytes(*s), lambda L, *s: L.fp8_linear_xent_workspace_bytes(*s, 0),
                                      lambda L, *s: L.fp8_linear_xent_workspace_bytes(*s, 1)], ids=["embedding", "loss", "loss_gradient"])
def test_workspaces_serve_smaller_calls(lib, bytes_of):
    r = random.Random(1)
    for _ in range(20000):
        T, V, D = int(2 ** r.uniform(0, 22)), int(2 ** r.uniform(0, 18)), 8 * int(2 ** r.uniform(0, 11))
        t, v, d = r.choice([r.randint(1, T), T]), r.choice([r.randint(1, V), V]), r.choice([8 * r.randint(1, D // 8), D])
        assert bytes_of(lib, t, v, d) <= bytes_of(lib, T, V, D), (t, v, d, T, V, D)


def test_binding_refuses_host_tensors():
    x, f = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(4)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        fg.linear_xent_fwd(x, x, i, f, f, x)
    with pytest.raises(ValueError):
        fg.embedding_fwd(i, x, x)
    with pytest.raises(ValueError):
        fg.rmsnorm_fwd_ckpt(x, x[0], 1e-5, fg.E4M3, x, x, f, f)
    with pytest.raises(ValueError):
        fg.swiglu_bwd_ckpt(x, f, x, fg.E4M3, x)
