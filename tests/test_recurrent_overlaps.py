"""Outputs over inputs that other blocks of a call still read are refused on the host, before anything is
enqueued (addresses as in tests/test_recurrent_args.py, never dereferenced)."""
import ctypes

import pytest

pytest.importorskip("torch")

from prefix_shared_chunkwise_gb300 import _lib as L
from tests.test_recurrent_args import EINVAL, LINEAR, _args


@pytest.fixture(scope="module", autouse=True)
def built():
    from prefix_shared_chunkwise_gb300 import build
    build.build()


@pytest.mark.parametrize("C", [1, 300])
@pytest.mark.parametrize("out", ["y", "z"])
@pytest.mark.parametrize("over", ["x", "weight", "bias"])
def test_linear_fwd_outputs_over_inputs(over, out, C):
    a = _args(L.LinearArgs, LINEAR, C=C, **{out: LINEAR[over]})
    assert L.lib().harts_linear_fwd(ctypes.byref(a), None) == EINVAL
    assert b"may not be" in L.lib().harts_last_error()
