"""The axes of the rotated pairs in the forms a caller may hold them, without a
GPU: a call that passes every check reaches the missing device."""

import numpy as np
import pytest
import torch

from test_rope_axes_host import PASSES, _built, _rope  # noqa: F401


def test_axes_in_any_form():
    axes = [0, 1, 2, 0] * 8
    for form in (bytes(axes), bytearray(axes), axes, tuple(axes), np.array(axes), np.array(axes, dtype=np.uint8),
                 np.array(axes, dtype=np.int32), torch.tensor(axes), torch.tensor(axes, dtype=torch.uint8),
                 (a for a in axes)):
        assert _rope(axis=form) == PASSES, type(form)
        if not hasattr(form, "__len__"):
            continue
        with pytest.raises(ValueError):
            _rope(axis=form[:-1])
    assert _rope(axis=np.array([3] * 32)) == -1   # an axis that positions do not have


@pytest.mark.parametrize("bad", [32, 64, 1.5, None, [0.0] * 32, ["0"] * 32])
def test_what_names_no_axes_is_refused(bad):
    with pytest.raises(TypeError):
        # (None: the default of _rope's own)
        _rope(axis=bad) if bad is not None else _rope(axis=[None] * 32)


def test_axes_past_a_byte():
    for bad in (256, -1):
        with pytest.raises(ValueError):
            _rope(axis=[bad] * 32)
