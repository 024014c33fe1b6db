"""What the Python side of the row passes does with its arguments, on a machine
without a GPU: tensors are stand-ins that are asked for their shape, type,
strides and address and never read."""
import pytest
import torch

from input_adaptive_block_b200 import api


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
