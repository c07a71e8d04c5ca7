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


def test_forward_mode_is_refused_with_grad_mode_off(monkeypatch):
    # the operators have no forward-mode derivative: a tangent may not vanish, whatever the
    # grad mode (the kernels' part is played by plain torch here)
    from torch.autograd import forward_ad
    monkeypatch.setattr(ops, "norm_forward", lambda x, w, b, eps, kind, save=False:
                        (x * 2, None, x.sum(-1)) if save else x * 2)
    monkeypatch.setattr(ops, "gated_ffn_forward", lambda x, W1, W3, W2, act, save=False:
                        (x * 2, x, x) if save else x * 2)
    monkeypatch.setattr(ops, "dropout_add_forward", lambda x, r, p, rng: x * 2)
    x, w = torch.ones(4, 8), torch.ones(8)
    calls = [lambda t: ops.layer_norm(t, w, w), lambda t: ops.rms_norm(t, w),
             lambda t: ops.layer_norm(x, t[0], w), lambda t: ops.layer_norm(x, w, t[0]),
             lambda t: ops.gated_ffn(t, x, x, x), lambda t: ops.gated_ffn(x, x, x, t),
             lambda t: ops.dropout_add(t, x, 0.0, None), lambda t: ops.dropout_add(x, t, 0.0, None),
             lambda t: ops.gated_ffn_block(t, x, x, x)]
    for call in calls:
        for mode in (torch.no_grad, torch.enable_grad):
            with mode(), forward_ad.dual_level():
                dual = forward_ad.make_dual(x, torch.ones_like(x))
                with pytest.raises((RuntimeError, NotImplementedError)):
                    call(dual)
        with torch.no_grad(), forward_ad.dual_level():
            assert torch.equal(call(x), x * 2) or call is calls[-1]
        with torch.no_grad():
            assert not call(x).requires_grad


def test_block_around_the_layer_refuses_gradients(monkeypatch):
    # forward only: a gradient or a tangent that is wanted may not be lost in silence (plain
    # torch plays the kernels' part)
    from torch.autograd import forward_ad

    from mixture_experts_ffn_expert_b200 import layer as layer_mod
    monkeypatch.setattr(layer_mod, "norm_forward", lambda x, w, b, eps, kind: x * 3)
    monkeypatch.setattr(layer_mod, "dropout_add_forward", lambda h, x, p, rng: h.detach() + x)
    layer = layer_mod.MoELayer.__new__(layer_mod.MoELayer)
    layer.forward = lambda h: h
    x, w = torch.ones(4, 8), torch.ones(8)
    out = layer.block(x, w)
    assert not out.requires_grad and torch.equal(out, x * 4)
    for wants in (0, 1):
        args = [x.clone(), w.clone()]
        args[wants].requires_grad_(True)
        out = layer.block(*args, p=0.1)
        assert out.requires_grad and torch.equal(out, x * 4)
        with pytest.raises(MoEError, match="no backward pass"):
            out.sum().backward()
        out = layer.block(*args)
        out += 1                                  # the result is the caller's, no view
        assert torch.equal(out, x * 4 + 1)
        with torch.no_grad():
            assert not layer.block(*args).requires_grad
    for mode in (torch.no_grad, torch.enable_grad):
        with mode(), forward_ad.dual_level(), pytest.raises(RuntimeError):
            layer.block(forward_ad.make_dual(x, torch.ones_like(x)), w)


def test_wait_timeout_hook_refuses_negative_launches():
    from mixture_experts_ffn_expert_b200.binding import load_library
    lib = load_library()
    assert lib.moe_ops_test_wait_timeout(-1) == 2
    assert lib.moe_ops_test_wait_timeout(0) == 0


def test_the_c_library_builds_without_torch_or_a_compiler(monkeypatch, capsys):
    # the C ABI does not need the torch module; ops.py without it raises (tested elsewhere)
    def no_compiler_runs(*a, **k):
        raise AssertionError("nothing may be compiled here")
    monkeypatch.setattr(build_mod.subprocess, "run", no_compiler_runs)
    real = build_mod.importlib.util.find_spec
    monkeypatch.setattr(build_mod.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else real(name, *a))
    assert build_mod.build() == build_mod.lib_path()
    assert "torch was not found" in capsys.readouterr().err
    monkeypatch.undo()
    monkeypatch.setenv("CXX", "no-such-compiler")
    assert build_mod.build() == build_mod.lib_path()
    assert "no-such-compiler was not found" in capsys.readouterr().err


def test_the_module_is_stale_when_torch_changes(monkeypatch):
    tag = build_mod._torch_tag()
    assert torch.__version__ in tag
    assert not build_mod._host_stale(build_mod.host_path(), tag)
    assert build_mod._host_stale(build_mod.host_path(), tag + "x")
