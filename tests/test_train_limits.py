"""The largest and smallest scale of the linear cross entropy's logits: the status before anything touches the GPU."""
import ctypes

import pytest

import fp8_fine_grained_x128_gb300 as fg
from fp8_fine_grained_x128_gb300 import build as fgbuild

P = 1 << 20            # a 16-byte aligned address that is never followed
S = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    fgbuild.build()
    return fg.lib()


# 2.4e38 log2 e is beyond FP32: the logits' factor would be infinite
@pytest.mark.parametrize("scale,status", [(2.0 ** 127, fg.OK), (1.8e38, fg.ERR_INVALID_ARG), (2.9e38, fg.ERR_INVALID_ARG), (1e-40, fg.OK)])
def test_scale(lib, scale, status):
    # no tokens: what is allowed does nothing
    assert lib.fp8_linear_xent_fwd(P, 0, 64, 64, P, 10, 64, P, scale, P, P, P, S) == status
    assert lib.fp8_linear_xent_bwd(P, 0, 64, 64, P, 10, 64, P, scale, P, P, P, P, P, 64, P, 1, 64, 1, P, S) == status
