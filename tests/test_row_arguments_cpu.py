"""What the Python side of the row passes does with its arguments, on a machine
without a GPU: tensors are stand-ins that are asked for their shape, type,
strides and address and never read."""
import ctypes

import pytest
import torch

from input_adaptive_block_b200 import _lib, api
from input_adaptive_block_b200._lib import (SPADE_ERR_INVALID, SPADE_ERR_WORKSPACE, SpadeRowDesc, SpadeRowGrads,
                                            SpadeRowParams)


class Standin:
    """A packed CUDA tensor as far as the argument checks look."""
    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, *shape, dtype=torch.bfloat16, at=1 << 40):
        self.shape, self.dtype, self.at = torch.Size(shape), dtype, at

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return self.at

    def stride(self, i=None):
        s = [self.shape[j + 1:].numel() for j in range(len(self.shape))]
        return tuple(s) if i is None else s[i]


def test_one_tensor_in_two_roles_has_its_shape_checked():
    """The tensor that the others are compared with is compared too: a
    gradient of Q given as K as well, with another number of heads."""
    t = Standin(10, 2, 64)
    assert api._strided(t, "k", t, (10, 2, 64), torch.bfloat16) == (1 << 40, 0)
    for shape in ((10, 5, 64), (10, 1, 64), (11, 2, 64)):
        for other in (t, Standin(10, 2, 64)):
            with pytest.raises(ValueError):
                api._strided(other, "k", t, shape, torch.bfloat16)
    with pytest.raises(TypeError):
        api._strided(t, "k", t, (10, 2, 64), torch.float32)


def test_scratch_is_for_parameter_gradients():
    """A backward call that wants none needs no workspace: the next check (dx
    over part of dh) refuses it, not the one of the workspace."""
    base, lib = 1 << 40, _lib.load()
    desc = SpadeRowDesc(rows=600, groups=1, dim=256, norm=2, eps=1e-6)
    for grads, ws, want in ((SpadeRowGrads(), None, SPADE_ERR_INVALID), (SpadeRowGrads(bias=9 * base), None, SPADE_ERR_WORKSPACE),
                            (SpadeRowGrads(), 8 * base, SPADE_ERR_WORKSPACE)):       # one that is given has its size
        got = lib.spade_norm_modulate_bwd(ctypes.byref(desc), ctypes.byref(SpadeRowParams()), base, None, 2 * base,
                                          base + 64, ctypes.byref(grads), ws, 16 if ws else 0, None)
        assert got == want, lib.spade_last_error_message()
    x, w = Standin(600, 256), Standin(256)
    none = dict.fromkeys(("gate", "post_weight", "weight", "bias", "scale", "shift"))
    assert api._row_scratch_bytes(x, desc, none) == 0
    assert api._row_scratch_bytes(x, desc, {**none, "bias": w}) == api.row_workspace_bytes(600, 256) > 0


def test_modulation_per_row_of_no_rows():
    """No rows and a modulation for each of them: no groups, nothing to do."""
    x, m = Standin(0, 64), Standin(0, 64)
    desc, params, _ = api._row_call(x, x.dtype, x.dtype, "layer", 1e-6, scale=m, shift=m)
    assert (desc.rows, desc.groups) == (0, 1) and not params.scale and not params.shift
    with pytest.raises(ValueError):
        api._row_call(Standin(5, 64), x.dtype, x.dtype, "layer", 1e-6, scale=m)


WIDE = 1 << 32


@pytest.mark.parametrize("call", [
    lambda x: api._row_call(Standin(1, WIDE + 64), x.dtype, x.dtype, "layer", 1e-6),
    lambda x: api._qk_desc(Standin(6, 1, WIDE + 64), None, None, None, (1, 2, 3), None, 0, 0, "none", 1e-6),
    lambda x: api._qk_desc(x, Standin(6, WIDE + 2, 64), None, None, (1, 2, 3), None, 0, 0, "none", 1e-6),
    lambda x: api._qk_desc(x, None, None, None, (1, WIDE + 2, 3), None, 0, 0, "none", 1e-6),
    lambda x: api._qk_desc(x, None, None, None, (1, 2, 3 - WIDE), None, 0, 0, "none", 1e-6),
    lambda x: api._qk_desc(x, None, None, None, (1, 2, 3), None, WIDE * WIDE, 0, "none", 1e-6),
    lambda x: api._qk_desc(x, None, None, None, (1, 2, 3), None, 0, WIDE * WIDE, "none", 1e-6),
    lambda x: api.rope_axes(8 * WIDE, (WIDE, 1, 1)),
    lambda x: api.row_workspace_bytes(600, WIDE + 256),
    lambda x: api.row_workspace_bytes(600, 256, WIDE * WIDE + 1),
    lambda x: api.qk_norm_rope_workspace_bytes(600, 4, WIDE + 4, 128, "head"),
])
def test_numbers_wider_than_the_descriptor(call):
    """Refused, not cut to their low bits."""
    with pytest.raises(ValueError, match="does not fit"):
        call(Standin(6, 2, 64))
