"""Pins of the operators' fp64 oracle, and the C ABI's refusals (host checks that return
before any CUDA call; no GPU needed)."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_expert_b200 import build as build_mod
from mixture_experts_ffn_expert_b200 import ops
from mixture_experts_ffn_expert_b200.binding import MoEError, load_library
from oracle import ops_oracle as O


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return load_library()


# ------------------------------------------------------------------------ oracle pins
@pytest.mark.parametrize("counter,key,want", [
    # the known answers published with the generator
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(counter, key, want):
    assert tuple(int(v) for v in O.philox_4x32_10(counter, key)) == want


def test_dropout_keep_share_and_independence():
    n = 1 << 18
    for p in (0.1, 0.5):
        k = O.dropout_keep(n, p, 5, 9)
        # a binomial share: six standard deviations
        assert abs(k.mean() - (1 - p)) < 6 * np.sqrt(p * (1 - p) / n)
    a, b = O.dropout_keep(n, 0.5, 5, 9), O.dropout_keep(n, 0.5, 5, 10)
    assert abs((a == b).mean() - 0.5) < 6 * 0.5 / np.sqrt(n)
    assert O.dropout_keep(10, 0.0, 1, 2).all() and not O.dropout_keep(10, 1.0, 1, 2).any()


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_oracle_against_torch_and_differences(kind):
    rng = np.random.default_rng(0)
    x, w, b = rng.normal(size=(5, 11)) + 0.5, rng.normal(size=11), rng.normal(size=11)
    y, _, _ = O.norm(x, w, b if kind == "layer" else None, 1e-3, kind)
    tx, tw, tb = (torch.tensor(v, dtype=torch.float64) for v in (x, w, b))
    if kind == "layer":
        want = torch.nn.functional.layer_norm(tx, (11,), tw, tb, 1e-3)
    else:
        want = torch.nn.functional.rms_norm(tx, (11,), tw, 1e-3)
    assert np.allclose(y, want.numpy(), rtol=1e-12, atol=1e-12)
    dy = rng.normal(size=x.shape)
    dx, dw, db = O.norm_grad(dy, x, w, 1e-3, kind)
    f = lambda xx, ww, bb: (O.norm(xx, ww, bb, 1e-3, kind)[0] * dy).sum()  # noqa: E731
    h = 1e-6
    for got, at, args in ((dx, x, 0), (dw, w, 1), (db, b, 2)):
        v = rng.normal(size=at.shape)
        hi, lo = [x, w, b], [x, w, b]
        hi[args], lo[args] = at + h * v, at - h * v
        assert abs((f(*hi) - f(*lo)) / (2 * h) - (got * v).sum()) < 1e-6


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_ffn_oracle_against_torch_and_differences(act):
    rng = np.random.default_rng(1)
    x, W1, W3 = rng.normal(size=(4, 6)), rng.normal(size=(5, 6)), rng.normal(size=(5, 6))
    W2, dout = rng.normal(size=(6, 5)), rng.normal(size=(4, 6))
    t = [torch.tensor(v, dtype=torch.float64) for v in (x, W1, W3, W2)]
    g = t[0] @ t[1].T
    a = torch.nn.functional.silu(g) if act == "silu" else \
        torch.nn.functional.gelu(g, approximate="tanh")
    want = (a * (t[0] @ t[2].T)) @ t[3].T
    assert np.allclose(O.gated_ffn(x, W1, W3, W2, act)[0], want.numpy(), rtol=1e-12)
    grads = O.gated_ffn_grad(dout, x, W1, W3, W2, act)
    at = [x, W1, W3, W2]
    h = 1e-6
    for i, got in enumerate(grads):
        v = rng.normal(size=at[i].shape)
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + h * v, at[i] - h * v
        diff = ((O.gated_ffn(*hi, act)[0] - O.gated_ffn(*lo, act)[0]) * dout).sum() / (2 * h)
        assert abs(diff - (got * v).sum()) < 1e-6 * max(1.0, abs(diff))


# ------------------------------------------------------------------------ refusals of the C ABI
P = 4096          # a non-null, aligned address; every call below returns before using it


def norm_args(**k):
    a = dict(kind=0, dtype=0, wdtype=0, rows=4, cols=64, x=P, ldx=64, weight=P, bias=None,
             eps=1e-5, y=P, ldy=64, mean=None, rstd=None, stream=None)
    a.update(k)
    return tuple(a.values())


@pytest.mark.parametrize("bad,status", [
    (dict(kind=2), 2), (dict(dtype=3), 2), (dict(dtype=0, wdtype=1), 2), (dict(rows=-1), 2),
    (dict(cols=0), 2), (dict(cols=(1 << 24) + 1), 5), (dict(rows=1 << 31), 5), (dict(x=None), 2),
    (dict(y=None), 2), (dict(ldx=63), 2), (dict(ldy=10), 2), (dict(x=P + 1), 2),
    (dict(weight=P + 1), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
    (dict(kind=1, bias=P), 2), (dict(kind=1, mean=P), 2), (dict(rstd=P + 2), 2),
])
def test_norm_forward_refuses(lib, bad, status):
    assert lib.moe_norm_forward(*norm_args(**bad)) == status
    assert lib.moe_last_error()


def norm_back_args(**k):
    a = dict(kind=0, dtype=0, wdtype=0, rows=4, cols=64, dy=P, lddy=64, x=P, ldx=64, weight=P,
             mean=P, rstd=P, dx=P, lddx=64, dweight=P, dbias=P, ws=P, nbytes=1 << 20, stream=None)
    a.update(k)
    return tuple(a.values())


@pytest.mark.parametrize("bad,status", [
    (dict(dy=None), 2), (dict(x=None), 2), (dict(rstd=None), 2), (dict(mean=None), 2),
    (dict(kind=1), 2), (dict(kind=1, mean=None), 2), (dict(lddy=1), 2), (dict(lddx=1), 2),
    (dict(ws=None), 2), (dict(ws=P + 4), 2), (dict(nbytes=2047), 3), (dict(dweight=P + 1), 2),
    (dict(dx=P + 1), 2),
])
def test_norm_backward_refuses(lib, bad, status):
    assert lib.moe_norm_backward(*norm_back_args(**bad)) == status


def test_norm_workspace_bytes(lib):
    assert lib.moe_norm_workspace_bytes(0, 4, 64) == 4 * 2 * 64 * 4
    assert lib.moe_norm_workspace_bytes(1, 4, 64) == 4 * 64 * 4
    assert lib.moe_norm_workspace_bytes(0, 10 ** 6, 64) == 296 * 2 * 64 * 4
    assert lib.moe_norm_workspace_bytes(7, 4, 64) == 0
    assert lib.moe_norm_workspace_bytes(0, -4, 64) == 0


def ffn_args(**k):
    a = dict(act=0, dtype=0, T=4, d=64, f=128, x=P, ldx=64, W1=P, W3=P, W2=P, out=P, ldo=64,
             gate=None, up=None, ws=P, nbytes=1 << 20, stream=None)
    a.update(k)
    return tuple(a.values())


@pytest.mark.parametrize("bad,status", [
    (dict(act=2), 2), (dict(dtype=2), 2), (dict(T=-1), 2), (dict(d=0), 1), (dict(f=0), 1),
    (dict(d=60), 5), (dict(f=4), 5), (dict(d=1 << 21), 5), (dict(T=(1 << 24) + 1), 5),
    (dict(x=None), 2), (dict(x=P + 8), 2), (dict(ldx=56), 2), (dict(ldx=68), 2),
    (dict(W1=None), 2), (dict(W3=P + 2), 2), (dict(W2=None), 2), (dict(out=None), 2),
    (dict(ldo=8), 2), (dict(gate=P), 2), (dict(gate=P, up=P + 8), 2), (dict(ws=None), 2),
    (dict(ws=P + 16), 2), (dict(nbytes=100), 3),
])
def test_gated_ffn_forward_refuses(lib, bad, status):
    assert lib.moe_gated_ffn_forward(*ffn_args(**bad)) == status


def ffn_back_args(**k):
    a = dict(act=0, dtype=0, T=4, d=64, f=128, dout=P, lddout=64, x=P, ldx=64, W1=P, W3=P, W2=P,
             gate=P, up=P, dx=P, lddx=64, dW1=P, dW3=P, dW2=P, ws=P, nbytes=1 << 20, stream=None)
    a.update(k)
    return tuple(a.values())


@pytest.mark.parametrize("bad,status", [
    (dict(act=-1), 2), (dict(dtype=2), 2), (dict(dout=None), 2), (dict(x=P + 8), 2),
    (dict(W1=None), 2), (dict(W3=None), 2), (dict(W2=None), 2), (dict(gate=None), 2),
    (dict(up=None), 2), (dict(dx=P + 2), 2), (dict(lddx=4), 2), (dict(dW1=P + 8), 2),
    (dict(dW2=P + 8), 2), (dict(ws=None), 2), (dict(nbytes=2048), 3), (dict(d=12), 5),
])
def test_gated_ffn_backward_refuses(lib, bad, status):
    assert lib.moe_gated_ffn_backward(*ffn_back_args(**bad)) == status


def drop_args(**k):
    a = dict(dtype=0, rows=4, cols=64, x=P, ldx=64, residual=P, ldr=64, p=0.1, rng=P, out=P,
             ldo=64, stream=None)
    a.update(k)
    return tuple(a.values())


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=5), 2), (dict(rows=-1), 2), (dict(cols=0), 2), (dict(p=-0.1), 2), (dict(p=1.1), 2),
    (dict(p=float("nan")), 2), (dict(x=None), 2), (dict(out=None), 2), (dict(rng=None), 2),
    (dict(rng=P + 4), 2), (dict(ldx=3), 2), (dict(ldr=3), 2), (dict(ldo=3), 2),
    (dict(x=P + 1), 2), (dict(rows=1 << 30, cols=1 << 20), 5),
])
def test_dropout_refuses(lib, bad, status):
    assert lib.moe_dropout_forward(*drop_args(**bad)) == status


def test_empty_batches_are_no_ops(lib):
    assert lib.moe_norm_forward(*norm_args(rows=0, x=None, y=None)) == 0
    assert lib.moe_gated_ffn_forward(*ffn_args(T=0)) == 0
    assert lib.moe_dropout_forward(*drop_args(rows=0)) == 0
    assert lib.moe_norm_backward(*norm_back_args(dx=None, dweight=None, dbias=None)) == 0
    assert lib.moe_gated_ffn_backward(*ffn_back_args(dx=None, dW1=None, dW3=None, dW2=None)) == 0


def test_cpu_tensors_are_refused():
    x, w = torch.zeros(4, 64), torch.zeros(64, 64)
    for call in (lambda: ops.norm_forward(x), lambda: ops.layer_norm(x), lambda: ops.rms_norm(x),
                 lambda: ops.gated_ffn(x, w, w, w),
                 lambda: ops.dropout_add(x, x, 0.1, torch.zeros(2, dtype=torch.int64)),
                 lambda: ops.dropout_add_backward(x, 0.1, None)):
        with pytest.raises(MoEError):
            call()


def test_missing_module_fails_loudly(monkeypatch, tmp_path):
    monkeypatch.setattr(ops, "_MODULE", None)
    monkeypatch.setattr(ops, "host_path", lambda: str(tmp_path / "nope.so"))
    with pytest.raises(MoEError):
        ops.norm_forward(torch.zeros(4, 64))
