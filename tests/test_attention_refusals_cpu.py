"""Calls of the attention sub-block that are refused, beyond those of
test_attention_cpu.py (nothing is launched)."""
import ctypes

import pytest

from test_attention_cpu import EINVAL, F16, attn, zp  # noqa: F401

FLT_MAX = (2 - 2.0 ** -23) * 2.0 ** 127


@pytest.mark.parametrize("backward", [False, True])
def test_a_scale_that_overflows_in_units_of_log_2_is_refused(zp, backward):  # noqa: F811
    """The kernels multiply scores by scale log2(e): infinity from FLT_MAX /
    log2(e) on, and then 0 for the largest score would be NaN."""
    s = zp.binding._Attention(4, 4, 1, 2, 1, 64, F16, 4, 0, 0.125, None, None, None)
    f = zp.binding._attention_lib().zero_window_attention_workspace_bytes
    for scale, ok in ((FLT_MAX, False), (FLT_MAX / 1.4, False), (FLT_MAX / 1.5, True), (1.0, True)):
        s.scale = scale
        assert (f(ctypes.byref(s), int(backward)) > 0) == ok, scale
        # (an accepted scale fails at the array, which is no device memory, with the same code)
        assert attn(zp, backward, scale=scale) == EINVAL


def test_a_rotarys_turns_are_not_set_behind_its_back(zp):  # noqa: F811
    """A call takes the address that the object was made with, so another
    tensor in its place would be read from memory that is gone."""
    import torch
    r = zp.Rotary([1.0, 0.5], interleaved=True, device="cpu")
    before, address = r.turns, r._c.turns
    assert (r.rot_dim, r.interleaved) == (4, True) and before.data_ptr() == address
    with pytest.raises(AttributeError):
        r.turns = torch.zeros_like(before)
    assert r.turns is before and r._c.turns == address
