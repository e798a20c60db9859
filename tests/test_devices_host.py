"""Tensors of a call that lie on another device than its queries, without a GPU: the kernels would
read them by an address that means nothing on theirs."""
import pytest
import torch

from exact_attention_126_b200 import fa


class OnDevice:
    """What the checks see of a contiguous tensor of some CUDA device."""

    def __init__(self, index, shape, dtype):
        self.shape, self.dtype, self.is_cuda = torch.Size(shape), dtype, True
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.device.index

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


CHECKS = {
    "alibi_slopes": ((4,), torch.float32, lambda t, q: fa._check_slopes(t, q)),
    "key_padding": ((2, 9), torch.bool, lambda t, q: fa._check_padding(t, q, 2, 9)),
    "seq_lengths": ((2,), torch.int32, lambda t, q: fa._check_lengths(t, q)),
    "cu_seqlens": ((3,), torch.int32, lambda t, q: fa._packed_dims(q, t, 9, None)),
    "prefix_lengths": ((2,), torch.int32, lambda t, q: fa._score(0.0, t, q, 2)),
}


@pytest.mark.parametrize("name", CHECKS)
def test_refused_on_another_device(name):
    shape, dtype, check = CHECKS[name]
    q = OnDevice(1, (18, 4, 64) if name == "cu_seqlens" else (2, 4, 9, 64), torch.bfloat16)
    check(OnDevice(1, shape, dtype), q)
    with pytest.raises(ValueError, match="device"):
        check(OnDevice(0, shape, dtype), q)
