"""What the operators' C calls refuse of the settings of their waits, and the binding of streams (nothing is
enqueued, so no GPU is needed)."""
from __future__ import annotations

import ctypes

import pytest

from rl_infra_gb300 import build, capi

ONE = 1 << 12          # a pointer that is never followed: each call is refused before a launch


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    capi.load()


@pytest.mark.parametrize("kw, said", [(dict(wait_limit_ms=10001), "wait_limit_ms"), (dict(withhold=17), "withhold"),
                                      (dict(d_status=ONE + 2), "misaligned")])
def test_scan_refuses_settings_of_its_waits(kw, said):
    sh = capi.per_scan_shape(steps=4, batch=2, channels=8, type=0, **kw)
    for n in ("h", "ga", "gx"):
        setattr(sh, "stride_" + n, (ctypes.c_int64 * 2)(32, 8))
    assert capi.per_scan_forward(ctypes.byref(sh), ONE, ONE, None, None, ONE, None, None) == capi.PER_ERR_INVALID_ARG
    assert said in capi.per_last_op_error()
    assert capi.per_scan_backward(ctypes.byref(sh), ONE, ONE, ONE, None, None, ONE, None, ONE, ONE, None, None) == \
        capi.PER_ERR_INVALID_ARG
    assert said in capi.per_last_op_error()


def test_binding_refuses_a_stream_of_another_device():
    """(It ran on the current stream of the tensors' device instead.)"""
    from rl_infra_gb300 import ops

    class Stream:
        device_index = 1

    with pytest.raises(ValueError, match="stream must be of cuda:0"):
        ops._On(Stream(), 0, (), None, None)
