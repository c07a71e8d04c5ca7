"""GPU edge cases of the norm, gated feed-forward and dropout operators: what the shapes and
values of the general tests do not reach. Bounds and helpers are those of the general tests
(u: half a step of a type, U32 = 2^-24)."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_expert_b200 import ops
from mixture_experts_ffn_expert_b200.binding import MoEError, load_library
from oracle import ops_oracle as O
from test_ops_edges_cpu import Wrapper
from test_ops_gpu import test_norm as base_norm
from test_ops_gpu import (DT, K, U32, check_ffn, close, drop_tol, f64, ffn_bounds, ffn_case, gen,
                          norm_bounds, randn, unit)

pytestmark = pytest.mark.gpu

# Rows and columns that reach every norm kernel: a warp and a block a row, aligned and not;
# tiles of many and of few rows, aligned and not; rows too long for registers.
NORM_KERNELS = [(5, 32), (3, 1000), (3, 1003), (2, 7168), (3, 70000), (700, 24), (700, 128),
                (700, 1000), (700, 1003), (700, 7168), (700, 7001), (1300, 16384), (601, 70000)]


# ------------------------------------------------------------------------ norm
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", NORM_KERNELS)
def test_constant_rows_have_their_value_as_mean(rows, cols, dtype):
    dt = DT[dtype]
    values = torch.tensor([1000.1, 123456.79, -0.1, 987.654, 1e8, 3.3, -1017.77, 0.0])
    if dtype == "fp16":
        values = values.clamp(-60000, 60000)
    v = values.to(dt).repeat((rows + 7) // 8)[:rows].cuda()
    x = v[:, None].expand(rows, cols).contiguous()
    b = randn(gen(1), cols, dtype=dt)
    y, mean, rstd = ops.norm_forward(x, None, b, save=True)
    assert torch.equal(mean, v.float())
    assert torch.equal(y, b.expand_as(y))
    # sqrt, division and eps itself: three roundings
    assert (rstd.double() * 1e-5 ** 0.5 - 1).abs().max().item() <= 4 * U32


@pytest.mark.parametrize("rows,cols", NORM_KERNELS)
def test_nearly_constant_rows(rows, cols):
    # Rows of a value plus 0 to 3 steps of it. The mean that a kernel may use is fp32: off by
    # half a step of it, U32 |mean|, and by its sum's error, relative to the rows' spread only.
    # It moves y by rstd times that, and the variance by its square.
    g = gen(rows + cols)
    values = torch.tensor([1000.1, 123456.79, -987.654, 33333.3]).repeat((rows + 3) // 4)[:rows]
    step = torch.from_numpy(np.spacing(np.abs(values.numpy())))
    x = values[:, None] + step[:, None] * torch.randint(0, 4, (rows, cols), generator=g)
    assert x.dtype == torch.float32
    y, mean, rstd = (f64(t) for t in ops.norm_forward(x.cuda(), save=True))
    x = x.double().numpy()
    want, m, r = O.norm(x)
    spread = x.max(1) - x.min(1)
    e = U32 * np.abs(m) * (1 + 2 * U32) + K * U32 * spread
    assert (np.abs(mean - m) <= e).all()
    # |d rstd| <= rstd^3 / 2 times the variance's error: e^2, and K U32 of the variance
    var = 1 / r ** 2 - 1e-5
    er = (e ** 2 + K * U32 * var) / (2 * (var + 1e-5)) + 4 * U32
    assert (np.abs(rstd / r - 1) <= er).all()
    xh = np.abs(want)
    tol = (r * e * (1 + er))[:, None] + xh * (er + 4 * U32)[:, None] + U32 * xh
    close(y, want, tol, "y")


@pytest.mark.parametrize("rows,cols", NORM_KERNELS)
def test_one_element_far_from_the_others(rows, cols):
    # A row's mean is summed as differences from the median p of three of its elements: it is off
    # by K U32 of the differences' mean size and by half a step of itself, which is small where p
    # is one of the ordinary elements, wherever the far one stands.
    g = gen(rows + 13 * cols)
    x = torch.randn((rows, cols), generator=g)
    far = [0, cols // 2, cols - 1, min(17, cols - 1)]
    for row in range(rows):
        x[row, far[row % 4]] = 1e6 * (1 - 2 * (row // 4 % 2))
    y, mean, rstd = (f64(t) for t in ops.norm_forward(x.cuda(), save=True))
    x = x.double().numpy()
    want, m, r = O.norm(x)
    p = np.median(x[:, [0, cols // 2, cols - 1]], axis=1)
    e = K * U32 * np.abs(x - p[:, None]).mean(1) + U32 * np.abs(m) * (1 + 2 * U32)
    assert (np.abs(mean - m) <= e).all()
    # the variance moves by e^2 and K U32 of itself
    er = (e * r) ** 2 / 2 + K * U32
    assert (np.abs(rstd / r - 1) <= er).all()
    close(y, want, (r * e)[:, None] + np.abs(want) * (er + 4 * U32)[:, None] + 1e-30, "y")


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("rows,cols", NORM_KERNELS)
def test_inverse_deviation_over_the_range(rows, cols, kind):
    # no eps: rows of any size from 1e-17 to 1e17, whose squares neither overflow nor leave
    # fp32's normal numbers; a statistic is off by K U32, the root and the division by 2 U32
    g = gen(rows + 3 * cols)
    scale = 10.0 ** (34.0 * torch.rand((rows, 1), generator=g) - 17.0)
    x = (torch.randn((rows, cols), generator=g) * scale).cuda()
    y, mean, rstd = ops.norm_forward(x, eps=0.0, kind=kind, save=True)
    want, m, r = O.norm(f64(x), eps=0.0, kind=kind)
    assert (np.abs(f64(rstd) / r - 1) <= K * U32).all()
    biggest = np.abs(f64(x)).max(axis=1, keepdims=True) if kind == "layer" else 0.0
    close(y, want, K * U32 * (np.abs(want) + r[:, None] * biggest), "y")


@pytest.mark.parametrize("rows,cols", [(3, 512), (3, 4096), (700, 128), (700, 1024), (1300, 512),
                                       (5000, 64), (2, 1 << 17)])
def test_inverse_root_of_exact_mean_squares(rows, cols):
    # rows of +-a, a of 8 bits: every sum of their squares is exact (a power of two of 16-bit
    # numbers), so the inverse deviation shows the root's and the division's roundings alone
    g = gen(rows + 7 * cols)
    a = torch.randint(128, 256, (rows, 1), generator=g) * \
        2.0 ** torch.randint(-60, 50, (rows, 1), generator=g)
    sign = 1 - 2 * torch.randint(0, 2, (rows, cols), generator=g)
    x = (a * sign).bfloat16().cuda()
    assert torch.equal(x.float().cpu().abs(), a.float().expand(rows, cols))
    rstd = f64(ops.norm_forward(x, eps=0.0, kind="rms", save=True)[2])
    assert np.abs(rstd * f64(a)[:, 0] - 1).max() <= 4 * U32


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("rows,cols", NORM_KERNELS)
def test_rows_that_are_not_finite_stay_alone(rows, cols, kind):
    """An infinity or a NaN in a row makes what IEEE arithmetic makes of the formulas, the same
    in every kernel, and leaves every other row's bits."""
    g = gen(rows + 5 * cols)
    x, dy = randn(g, rows, cols, dtype=torch.float32), randn(g, rows, cols, dtype=torch.float32)
    w = randn(g, cols, dtype=torch.float32, shift=1.0)
    b = randn(g, cols, dtype=torch.float32) if kind == "layer" else None
    inf, nan = float("inf"), float("nan")
    clean = ops.norm_forward(x, w, b, kind=kind, save=True)
    for col in (0, cols // 2, cols - 1):
        for value in (inf, -inf, nan):
            bad = rows // 2
            x2 = x.clone()
            x2[bad, col] = value
            y, mean, rstd = ops.norm_forward(x2, w, b, kind=kind, save=True)
            dx, dw, db = ops.norm_backward(dy, x2, w, mean, rstd, kind=kind, bias=b is not None)
            keep = torch.arange(rows, device="cuda") != bad
            assert torch.equal(y[keep], clean[0][keep]) and torch.equal(rstd[keep], clean[2][keep])
            dx0 = ops.norm_backward(dy, x, w, clean[1], clean[2], kind=kind)[0]
            assert torch.equal(dx[keep], dx0[keep])
            assert torch.isnan(dx[bad]).all()
            if kind == "layer":
                assert torch.equal(mean[keep], clean[1][keep])
                # x - infinity: no row without a NaN
                assert torch.equal(mean[bad].cpu(), torch.tensor(value)) or value != value
                assert value == value or torch.isnan(mean[bad])
                assert torch.isnan(rstd[bad]) and torch.isnan(y[bad]).all()
                assert torch.isnan(dw).all() and torch.isfinite(db).all()
            elif value == value:
                # the mean square is infinite: 1 / sqrt = 0, 0 for finite elements
                assert rstd[bad] == 0 and torch.isnan(y[bad, col])
                others = torch.arange(cols, device="cuda") != col
                assert (y[bad, others] == 0).all()
                assert torch.isnan(dw[col]) and torch.isfinite(dw[others]).all()
            else:
                assert torch.isnan(rstd[bad]) and torch.isnan(y[bad]).all()
                assert torch.isnan(dw).all()


# ------------------------------------------------------------------------ arguments
def test_an_argument_without_memory_is_not_an_absent_one():
    x, W1, W3, W2, dout = ffn_case(8, 64, 72, "bf16", 40)
    out, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, save=True)
    y, mean, rstd = ops.norm_forward(x, save=True)
    w = torch.ones(64, device="cuda")
    rng = torch.tensor([1, 2], device="cuda")
    wrap = lambda t: Wrapper(t, t.device)                                  # noqa: E731
    calls = [lambda: ops.norm_forward(x, wrap(w)), lambda: ops.norm_forward(x, w, wrap(w)),
             lambda: ops.norm_forward(x, None, wrap(w)),
             lambda: ops.norm_backward(dout, x, wrap(w), mean, rstd),
             lambda: ops.norm_backward(wrap(dout), x, w, mean, rstd),
             lambda: ops.norm_backward(dout, x, w, wrap(mean), rstd),
             lambda: ops.norm_backward(dout, x, w, mean, wrap(rstd)),
             lambda: ops.dropout_add_forward(x, wrap(dout), 0.1, rng),
             lambda: ops.dropout_add_forward(x, wrap(dout), 0.0, None),
             lambda: ops.dropout_add_forward(x, dout, 0.1, wrap(rng)),
             lambda: ops.gated_ffn_forward(x, wrap(W1), W3, W2),
             lambda: ops.gated_ffn_forward(x, W1, W3, wrap(W2)),
             lambda: ops.gated_ffn_backward(dout, x, W1, W3, W2, wrap(gate), up),
             lambda: ops.gated_ffn_backward(wrap(dout), x, W1, W3, W2, gate, up)]
    for i, call in enumerate(calls):
        with pytest.raises(MoEError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_negated_rng_is_refused():
    # torch's negative bit: memory holds the unnegated seed and offset
    x = randn(gen(41), 6, 64)
    rng = torch.tensor([5, 6], device="cuda")
    neg = torch._neg_view(rng)
    with pytest.raises(MoEError):
        ops.dropout_add_forward(x, x, 0.5, neg)
    with pytest.raises(MoEError):
        ops.dropout_add_backward(x, 0.5, neg)
    want = ops.dropout_add_forward(x, x, 0.5, torch.tensor([-5, -6], device="cuda"))
    assert torch.equal(ops.dropout_add_forward(x, x, 0.5, neg.resolve_neg()), want)


def test_forward_mode_is_refused_with_grad_mode_off():
    from torch.autograd import forward_ad
    x, W1, W3, W2, _ = ffn_case(8, 64, 72, "bf16", 42)
    rng = torch.tensor([1, 2], device="cuda")
    want = ops.gated_ffn_block(x, W1, W3, W2, p=0.25, rng=rng)
    with torch.no_grad(), forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        dual_w = forward_ad.make_dual(W3, torch.ones_like(W3))
        for call in (lambda: ops.rms_norm(dual), lambda: ops.layer_norm(dual),
                     lambda: ops.gated_ffn(dual, W1, W3, W2), lambda: ops.gated_ffn(x, W1, dual_w, W2),
                     lambda: ops.dropout_add(x, dual, 0.25, rng),
                     lambda: ops.gated_ffn_block(dual, W1, W3, W2, p=0.25, rng=rng)):
            with pytest.raises(RuntimeError, match="forward mode|jvp"):
                call()
        assert torch.equal(ops.gated_ffn_block(x, W1, W3, W2, p=0.25, rng=rng), want)


def test_block_around_the_layer_refuses_gradients():
    from mixture_experts_ffn_expert_b200.inputs import WORKLOADS, make_layer_inputs
    from mixture_experts_ffn_expert_b200.layer import MoELayer
    s = WORKLOADS["tiny_t256_d128_f64_e31k7_s1"]
    inp = make_layer_inputs(s, seed=0, device="cuda")
    layer = MoELayer(s.d, s.f, s.n_routed, s.top_k, s.n_shared, s.renorm, inp, bias=inp["bias"])
    w = randn(gen(43), s.d, scale=0.1, shift=1.0)
    rng = torch.tensor([1, 2], device="cuda")
    want = layer.block(inp["x"], w, p=0.1, rng=rng)
    assert not want.requires_grad
    for x, v in ((inp["x"].clone().requires_grad_(True), w),
                 (inp["x"], w.clone().requires_grad_(True))):
        out = layer.block(x, v, p=0.1, rng=rng)
        assert torch.equal(out, want)
        with pytest.raises(MoEError, match="no backward pass"):
            out.sum().backward()
        with torch.no_grad():
            assert not layer.block(x, v, p=0.1, rng=rng).requires_grad


# ------------------------------------------------------------------------ C interface
def stream():
    return torch.cuda.current_stream().cuda_stream


def padded(rows, cols, pad, dtype):
    """An output whose rows are cols + pad apart, filled with a sentinel, and its view."""
    buf = torch.full((rows, cols + pad), 7.0, dtype=dtype, device="cuda")
    return buf, buf[:, :cols]


def padding_kept(buf, cols):
    return torch.equal(buf[:, cols:], torch.full_like(buf[:, cols:], 7.0))


@pytest.mark.parametrize("pad", [8, 5])
@pytest.mark.parametrize("rows,cols", NORM_KERNELS)
def test_norm_padded_outputs(rows, cols, pad):
    lib = load_library()
    g = gen(rows + 9 * cols)
    x, dy = randn(g, rows, cols), randn(g, rows, cols)
    w, b = randn(g, cols, shift=1.0), randn(g, cols)
    y, mean, rstd = ops.norm_forward(x, w, b, save=True)
    buf, view = padded(rows, cols, pad, x.dtype)
    assert lib.moe_norm_forward(0, 0, 0, rows, cols, x.data_ptr(), cols, w.data_ptr(),
                                b.data_ptr(), 1e-5, buf.data_ptr(), cols + pad, None, None,
                                stream()) == 0
    want = norm_bounds(f64(x), f64(w), f64(b), f64(dy), x.dtype, x.dtype, "layer", 1e-5)
    close(view, *want[0], "y")
    assert padding_kept(buf, cols)
    buf, view = padded(rows, cols, pad, x.dtype)
    dw2, db2 = torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(lib.moe_norm_workspace_bytes(0, rows, cols), dtype=torch.uint8, device="cuda")
    assert lib.moe_norm_backward(0, 0, 0, rows, cols, dy.data_ptr(), cols, x.data_ptr(), cols,
                                 w.data_ptr(), mean.data_ptr(), rstd.data_ptr(), buf.data_ptr(),
                                 cols + pad, dw2.data_ptr(), db2.data_ptr(), ws.data_ptr(),
                                 ws.numel(), stream()) == 0
    for name, got, (ref, tol) in zip(("dx", "dweight", "dbias"), (view, dw2, db2), want[1:]):
        close(got, ref, tol, name)
    assert padding_kept(buf, cols)


# streamed, single CTAs, split reductions beyond a token tile, pairs
FFN_KERNELS = [(1, 136, 264), (40, 136, 264), (100, 520, 520), (128, 1024, 1024), (300, 136, 264),
               (333, 2048, 1408), (2321, 2088, 2632)]


@pytest.mark.parametrize("T,d,f", FFN_KERNELS)
def test_gated_ffn_padded_tensors(T, d, f):
    lib = load_library()
    x, W1, W3, W2, dout = ffn_case(T, d, f, "bf16", 44)
    out, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, save=True)
    grads = ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up)
    ld = d + 24
    wide = lambda t: torch.cat([t, torch.full((T, 24), float("nan"), device="cuda",  # noqa: E731
                                              dtype=t.dtype)], 1)
    xw, dw = wide(x), wide(dout)
    ws = torch.empty(lib.moe_gated_ffn_workspace_bytes(T, d, f, 1), dtype=torch.uint8,
                     device="cuda")
    buf, view = padded(T, d, 24, x.dtype)
    P = lambda *ts: [t.data_ptr() for t in ts]                             # noqa: E731
    assert lib.moe_gated_ffn_forward(0, 0, T, d, f, xw.data_ptr(), ld, *P(W1, W3, W2, buf), ld,
                                     None, None, ws.data_ptr(), ws.numel(), stream()) == 0
    assert torch.equal(view, out) and padding_kept(buf, d)
    buf, view = padded(T, d, 24, x.dtype)
    mine = [torch.empty_like(t) for t in grads[1:]]
    assert lib.moe_gated_ffn_backward(0, 0, T, d, f, dw.data_ptr(), ld, xw.data_ptr(), ld,
                                      *P(W1, W3, W2, gate, up, buf), ld, *P(*mine), ws.data_ptr(),
                                      ws.numel(), stream()) == 0
    assert torch.equal(view, grads[0]) and padding_kept(buf, d)
    assert all(torch.equal(a, b) for a, b in zip(mine, grads[1:]))
    # dx alone: its own launch of another kernel for few tokens
    buf, view = padded(T, d, 24, x.dtype)
    assert lib.moe_gated_ffn_backward(0, 0, T, d, f, dw.data_ptr(), ld, xw.data_ptr(), ld,
                                      *P(W1, W3, W2, gate, up, buf), ld, None, None, None,
                                      ws.data_ptr(), ws.numel(), stream()) == 0
    alone = ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up,
                                   needs=(True, False, False, False))[0]
    assert torch.equal(view, alone) and padding_kept(buf, d)
    want, tol = ffn_bounds(*(f64(t) for t in (x, W1, W3, W2, dout)), "silu", x.dtype)["dx"]
    close(alone, want, tol, "dx alone")
    ops.device_status()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (33, 128), (777, 1001)])
def test_dropout_c_interface(rows, cols, dtype):
    lib = load_library()
    g = gen(rows + 11 * cols)
    dt = DT[dtype]
    code = {"bf16": 0, "fp32": 2}[dtype]
    x, res = randn(g, rows, cols, dtype=dt), randn(g, rows, cols, dtype=dt)
    rng = torch.tensor([31, 32], device="cuda")
    p = 0.3
    out = ops.dropout_add_forward(x, res, p, rng)
    want = O.dropout_add(f64(x), None, p, 31, 32)
    dx = torch.empty_like(x)
    assert lib.moe_dropout_backward(code, rows, cols, x.data_ptr(), cols, p, rng.data_ptr(),
                                    dx.data_ptr(), cols, stream()) == 0
    close(dx, want, drop_tol(f64(x), None, p, dt, want), "dx")
    # in place: over dout, over x, over the residual
    for over in ("dout", "x", "residual"):
        a, r = x.clone(), res.clone()
        target = r if over == "residual" else a
        if over == "dout":
            assert lib.moe_dropout_backward(code, rows, cols, a.data_ptr(), cols, p,
                                            rng.data_ptr(), a.data_ptr(), cols, stream()) == 0
            assert torch.equal(a, dx)
            continue
        assert lib.moe_dropout_forward(code, rows, cols, a.data_ptr(), cols, r.data_ptr(), cols, p,
                                       rng.data_ptr(), target.data_ptr(), cols, stream()) == 0
        assert torch.equal(target, out) and torch.equal(r if over == "x" else a,
                                                        res if over == "x" else x)
    # padded outputs, and in place with padding (strided kernels)
    for pad in (8, 5):
        buf, view = padded(rows, cols, pad, dt)
        assert lib.moe_dropout_forward(code, rows, cols, x.data_ptr(), cols, res.data_ptr(), cols, p,
                                       rng.data_ptr(), buf.data_ptr(), cols + pad, stream()) == 0
        assert torch.equal(view, out) and padding_kept(buf, cols)
        view.copy_(x)
        assert lib.moe_dropout_forward(code, rows, cols, buf.data_ptr(), cols + pad,
                                       res.data_ptr(), cols, p, rng.data_ptr(), buf.data_ptr(),
                                       cols + pad, stream()) == 0
        assert torch.equal(view, out) and padding_kept(buf, cols)
        buf, view = padded(rows, cols, pad, dt)
        assert lib.moe_dropout_backward(code, rows, cols, x.data_ptr(), cols, p, rng.data_ptr(),
                                        buf.data_ptr(), cols + pad, stream()) == 0
        assert torch.equal(view, dx) and padding_kept(buf, cols)


# ------------------------------------------------------------------------ failure path
def norm_call(rows, cols, backward):
    g = gen(rows + cols)
    x, dy = randn(g, rows, cols), randn(g, rows, cols)
    w = randn(g, cols, shift=1.0)
    _, mean, rstd = ops.norm_forward(x, w, save=True)
    if backward:
        return lambda: ops.norm_backward(dy, x, w, mean, rstd)[:2]
    return lambda: (ops.norm_forward(x, w),)


def ffn_call(T, d, f, needs=None):
    x, W1, W3, W2, dout = ffn_case(T, d, f, "bf16", 45)
    _, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, save=True)
    if needs:
        return lambda: [t for t in ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up,
                                                          needs=needs) if t is not None]
    return lambda: (ops.gated_ffn_forward(x, W1, W3, W2),)


ALL, DX = (True,) * 4, (True, False, False, False)


@pytest.mark.parametrize("make,launch", [
    (lambda: norm_call(700, 1000, False), 1), (lambda: norm_call(700, 1003, False), 1),
    (lambda: norm_call(700, 1000, True), 1), (lambda: norm_call(3000, 128, True), 1),
    (lambda: ffn_call(1, 136, 2048), 1), (lambda: ffn_call(24, 2048, 1408), 2),
    (lambda: ffn_call(100, 2048, 2816), 1), (lambda: ffn_call(40, 2048, 1408, DX), 2),
    (lambda: ffn_call(128, 1024, 1024), 1), (lambda: ffn_call(128, 1024, 1024), 2),
    (lambda: ffn_call(300, 136, 264, ALL), 2),
    (lambda: ffn_call(2321, 2088, 2632), 1), (lambda: ffn_call(2321, 2088, 2632, ALL), 1),
    (lambda: ffn_call(2321, 2088, 2632, ALL), 2),
], ids=["norm", "norm_odd", "norm_backward", "norm_backward_short", "stream", "stream_early",
        "stream_128", "stream_dx_early", "single", "single_down", "single_gradients", "pairs",
        "pairs_dh", "pairs_gradients"])
def test_a_wait_that_runs_out_is_reported_and_the_context_recovers(make, launch):
    """The failure path without a fault: one block withholds its first copy, the bounded waits
    for it run out (2 s), the kernel reports and returns; the next call has its usual bits."""
    import time
    lib = load_library()
    call = make()
    want = [t.clone() for t in call()]
    ops.device_status()
    assert lib.moe_ops_test_wait_timeout(launch) == 0
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    waited = time.perf_counter() - t0
    assert lib.moe_ops_test_wait_timeout(0) == 0
    with pytest.raises(MoEError) as e:
        ops.device_status()
    assert e.value.status == 6                     # MOE_DEVICE_TIMEOUT
    ops.device_status()                            # reading cleared it
    assert 1.5 < waited < 30.0, waited             # bounded waits, not a hang
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    ops.device_status()


# ------------------------------------------------------------------------ gated feed-forward
@pytest.mark.parametrize("T", [3, 200, 2321])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_gates_beyond_their_range_have_their_gradient(T, act, dtype):
    # One hidden column has gates of -98304, beyond fp16, or (bf16) of -2^70, whose square is not
    # in fp32. act and act' are 0 there as they are at -200, so every result has the bits that
    # gates of -200 give; at the opposite gates act' is 1 as at 200.
    d, f = (72, 136) if T < 2321 else (2088, 2632)
    x, W1, W3, W2, dout = ffn_case(T, d, f, dtype, 46)
    first, big = (2.0, 98304.0) if dtype == "fp16" else (2.0 ** 35, 2.0 ** 70)
    x[:, 0] = first
    W1[:, 0], W3[:, 0], W1[5] = 0, 0, 0

    def step(gate_value, needs):
        W1[5, 0] = gate_value / first
        out, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, act, save=True)
        assert gate.dtype == up.dtype == torch.float32 and (gate[:, 5] == gate_value).all()
        return [out, *ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up, act, needs)]

    near = 200.0 if dtype == "fp16" else 2.0 ** 8
    for a, b in zip(step(-big, (False, True, True, True)), step(-near, (False, True, True, True))):
        assert a is b is None or (torch.isfinite(a).all() and torch.equal(a, b))
    far, ref = step(big, (False, True, False, False)), step(near, (False, True, False, False))
    assert torch.isfinite(far[2]).all() and torch.equal(far[2], ref[2])
    # dx: the column's dgate and dup are 0, its weights finite
    dx = step(-big, (True, False, False, False))[1]
    assert torch.isfinite(dx).all()
    W1[5, 0] = 0
    gate, up = ops.gated_ffn_forward(x, W1, W3, W2, act, save=True)[1:]
    for infinite in (-float("inf"), -near):          # the limit, and as at -200
        gate[:, 5] = infinite
        W1[5, 0] = -big / first
        assert torch.equal(dx, ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up, act,
                                                      (True, False, False, False))[0])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,d,f", [(24, 2048, 2816), (100, 520, 520), (333, 2048, 1408),
                                   (2321, 2088, 2632)])
def test_gradients_have_one_rounding_beside_their_own(T, d, f, dtype, act):
    # out, dW and dx each round one operand of their last product (h, dgate, dup) and the result:
    # two roundings of one size that do not know of each other, sqrt(2) of what rounding the exact
    # result gives; 1.5 leaves 6% for the reductions' fp32
    x, W1, W3, W2, dout = ffn_case(T, d, f, dtype, 51)
    out, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, act, save=True)
    assert gate.dtype == up.dtype == torch.float32
    got = [out, *ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up, act)]
    ax, a1, a3, a2, ad = (f64(t) for t in (x, W1, W3, W2, dout))
    want = [O.gated_ffn(ax, a1, a3, a2, act)[0], *O.gated_ffn_grad(ad, ax, a1, a3, a2, act)]
    for name, t, ref in zip(("out", "dx", "dW1", "dW3", "dW2"), got, want):
        rounded = f64(torch.from_numpy(ref).to(t.dtype))
        off, once = np.linalg.norm(f64(t) - ref), np.linalg.norm(rounded - ref)
        assert off <= 1.5 * once, f"{name}: {off / once} roundings"


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(100001, 1), (60000, 3), (50000, 8), (30011, 17), (9000, 40)])
def test_norm_many_short_rows(rows, cols, dtype):
    base_norm(rows, cols, dtype, dtype, "layer")
    base_norm(rows, cols, dtype, "fp32", "rms")


@pytest.mark.parametrize("cols", [8192, 8191])
def test_norm_beyond_32_bits(cols):
    # 4.9e9 elements; the gradient of the weights comes from a few rows, the others' dy is 0
    rows = 600_000
    torch.manual_seed(0)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_()
    at = [0, 1, 299_999, 524_288, 524_289, rows - 2, rows - 1]
    dy = torch.zeros_like(x)
    some = randn(gen(47), len(at), cols)
    dy[at] = some
    w = randn(gen(48), cols, shift=1.0)
    y, mean, rstd = ops.norm_forward(x, w, save=True)
    want = norm_bounds(f64(x[at]), f64(w), None, f64(some), x.dtype, x.dtype, "layer", 1e-5)
    close(y[at], *want[0], "y")
    del y
    dx, dw, db = ops.norm_backward(dy, x, w, mean, rstd, bias=True)
    close(dx[at], *want[1], "dx")
    close(dw, *want[2], "dweight")
    close(db, *want[3], "dbias")
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[at] = False
    assert dx.abs().amax(1)[keep].max() == 0


@pytest.mark.parametrize("T,d,f,dtype,act", [
    (100_003, 8, 8, "bf16", "silu"), (40_000, 64, 16, "fp16", "gelu"), (3, 16384, 8, "bf16", "gelu"),
    (130, 8, 16384, "fp16", "silu"), (257, 20000, 24, "bf16", "silu"), (1, 8, 30000, "bf16", "silu"),
    (4099, 8, 1000, "bf16", "gelu")])
def test_gated_ffn_lopsided_shapes(T, d, f, dtype, act):
    check_ffn(T, d, f, dtype, act)


def test_gated_ffn_beyond_32_bits():
    # 4.3e9 hidden elements; gradients from a few tokens, the others' dout is 0
    T, d, f = 300_001, 64, 14336
    x, W1, W3, W2, _ = ffn_case(8, d, f, "bf16", 49)
    at = [0, 1, 127, 149_999, 299_000, 299_592, T - 2, T - 1]
    torch.manual_seed(1)
    xl = torch.empty((T, d), dtype=torch.bfloat16, device="cuda").normal_()
    xl[at] = x
    dout = torch.zeros_like(xl)
    some = randn(gen(50), 8, d, scale=0.25)
    dout[at] = some
    out, gate, up = ops.gated_ffn_forward(xl, W1, W3, W2, save=True)
    grads = ops.gated_ffn_backward(dout, xl, W1, W3, W2, gate, up)
    ops.device_status()
    want = ffn_bounds(*(f64(t) for t in (x, W1, W3, W2, some)), "silu", x.dtype)
    close(out[at], *want["out"], "out")
    close(grads[0][at], *want["dx"], "dx")
    # T products a reduction, of which 8 are not 0: adding zeros rounds nothing
    for name, got in zip(("dW1", "dW3", "dW2"), grads[1:]):
        close(got, *want[name], name)


def test_dropout_refuses_its_probability_for_empty_tensors_too():
    x = torch.zeros((0, 8), device="cuda")
    rng = torch.tensor([1, 2], device="cuda")
    for p in (-0.5, 1.5, float("nan")):
        with pytest.raises(MoEError):
            ops.dropout_add_forward(x, None, p, rng)
    assert ops.dropout_add_forward(x, None, 0.5, rng).shape == (0, 8)
