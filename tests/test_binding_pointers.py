"""What the binding takes for a pointer, and that raw pointers and None do not go by way of an exception."""

import enum
import sys

import numpy as np
import pytest
import torch

from mxfp4_a4w4_gemm_gb300 import _native


def raises(fn, *args):
    """Exceptions raised while fn runs, caught ones too."""
    seen, tool = [], sys.monitoring.DEBUGGER_ID
    sys.monitoring.use_tool_id(tool, "test_binding_pointers")
    try:
        sys.monitoring.register_callback(tool, sys.monitoring.events.RAISE, lambda code, at, e: seen.append(e))
        sys.monitoring.set_events(tool, sys.monitoring.events.RAISE)
        got = fn(*args)
    finally:
        sys.monitoring.set_events(tool, 0)
        sys.monitoring.free_tool_id(tool)
    return got, seen


@pytest.mark.parametrize("fn", [lambda x: _native._ptr(x), lambda x: _native._rows_ptr(x, 64)])
@pytest.mark.parametrize("x", [None, 0, 4096, 2 ** 47 + 16])
def test_raw_pointers_pass_without_an_exception(fn, x):
    got, seen = raises(fn, x)
    assert got == x and seen == []


class Address(enum.IntEnum):
    HERE = 512


def test_what_is_a_pointer():
    t = torch.zeros(4, 6)
    assert _native._ptr(t) == t.data_ptr() and _native._ptr(t[1:]) == t[1:].data_ptr() and _native._ptr(Address.HERE) == 512
    for bad in (t[:, 1:], t.t()):
        with pytest.raises(ValueError):
            _native._ptr(bad)
    for bad in (np.zeros(4), "x", 1.5, [1]):
        with pytest.raises(TypeError):
            _native._ptr(bad)


def test_rows_may_be_slices():
    t = torch.zeros(5, 6, 8)
    assert _native._rows_ptr(t[:, 2:4], 48) == t.data_ptr() + 2 * 8 * 4
    assert _native._rows_ptr(t.view(5, 48), 48) == t.data_ptr() and _native._rows_ptr(t[:1, 1:], 7) == t.data_ptr() + 8 * 4
    for bad, stride in ((t[:, 2:4], 16), (t[:, :, 1:], 48), (t[:, ::2], 48), (t[:, 0, :4], 8)):
        with pytest.raises(ValueError):
            _native._rows_ptr(bad, stride)
