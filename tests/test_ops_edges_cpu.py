"""Refusals of the operators' torch functions that need no GPU."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from mixture_experts_ffn_expert_b200 import build as build_mod
from mixture_experts_ffn_expert_b200 import ops
from mixture_experts_ffn_expert_b200.binding import MoEError


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


class Wrapper(torch.Tensor):
    """A tensor that says it is on a device and holds another one instead of memory."""

    @staticmethod
    def __new__(cls, inner, device):
        return torch.Tensor._make_wrapper_subclass(cls, inner.shape, dtype=inner.dtype,
                                                   device=device)

    def __init__(self, inner, device):
        self.inner = inner

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(str(func))


def fake(*shape):
    with FakeTensorMode():
        return torch.empty(shape, device="cuda")


@pytest.mark.parametrize("make", [lambda: Wrapper(torch.ones(4, 64), "cuda:0"),
                                  lambda: fake(4, 64)], ids=["wrapper", "fake"])
def test_tensors_without_memory_are_refused(make):
    t = make()
    assert t.is_cuda
    for call in (lambda: ops.norm_forward(t), lambda: ops.gated_ffn_forward(t, t, t, t),
                 lambda: ops.norm_backward(t, t, None, None, t),
                 lambda: ops.gated_ffn_backward(t, t, t, t, t, t, t),
                 lambda: ops.dropout_add_forward(t, None, 0.0, None)):
        with pytest.raises(MoEError, match="no memory of its own"):
            call()
