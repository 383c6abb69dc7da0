"""The answering side's Python calls on the host: what they refuse before any
work, and what they must not do to the process."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from sequence_sparse_attention_b200 import RopeLayout
from sequence_sparse_attention_b200.cache import _load_calls


# ------------------------------------------------------------------ tensors without memory
@pytest.mark.parametrize("transform", ["vmap", "grad", "none"])
def test_tensors_without_memory_are_refused(transform):
    """Inside torch.func's transforms a tensor has no address to take, nor has one
    of a FakeTensorMode: the call raises (and does not end the process), before it
    looks for a device."""
    cfg = RopeLayout(4, 2, 64).c()
    rope = _load_calls().Rope(ctypes.addressof(cfg), 0, 0, 0, 0)
    with FakeTensorMode():
        q, k, qo, ko = (torch.empty(2, h, 64, dtype=torch.bfloat16, device="cuda:0") for h in (4, 2, 4, 2))
        pos = torch.empty(1, 2, dtype=torch.int32, device="cuda:0")
        with pytest.raises((RuntimeError, ValueError), match="data pointer|storage|memory"):
            if transform == "vmap":
                torch.vmap(lambda x: rope.apply(x, k, pos, qo, ko))(torch.stack([q] * 3))
            elif transform == "grad":
                torch.func.grad(lambda x: rope.apply(x, k, pos, qo, ko)[0].float().sum())(q)
            else:
                rope.apply(q, k, pos, qo, ko)
