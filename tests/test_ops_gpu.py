"""GPU parity of the norm, gated feed-forward and dropout operators against the fp64 oracle.

Tolerances are forward error bounds, element by element, computed from the oracle's
quantities. u is half a step of the output's type (bf16 2^-8, fp16 2^-11, fp32 2^-24) and
counts every rounding to it; U32 = 2^-24 counts fp32 arithmetic. A sum of n terms that a
kernel adds in chains of at most c terms is off by at most c * U32 times the sum of the
magnitudes; the norm kernels' chains (elements a thread holds or strides over, plus two
shuffle trees) are at most 110 for the sizes below, so K = 128 bounds a statistic.
"""
import math

import numpy as np
import pytest
import torch

from mixture_experts_ffn_expert_b200 import ops
from mixture_experts_ffn_expert_b200.binding import MoEError, load_library
from oracle import ops_oracle as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U32 = 2.0 ** -24
K = 128


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    # half the spacing of the type's subnormals (bf16 and fp32: far below any value here)
    return 2.0 ** -25 if dtype == torch.float16 else 1e-37


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(gen, *shape, dtype=torch.bfloat16, scale=1.0, shift=0.0):
    v = torch.randn(shape, generator=gen, dtype=torch.float32)
    return (v * scale + shift).to(dtype).cuda()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(got, want, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - want) - tol
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over[i] <= 0, f"{what}: at {i} got {got[i]} want {want[i]} tolerance {tol[i]}"


# ------------------------------------------------------------------------ norm
def norm_bounds(x, w, b, dy, dtype, wdtype, kind, eps):
    """(y, tol), and with dy also (dx, tol), (dw, tol), (db, tol)."""
    u = unit(dtype)
    y, mean, rstd = O.norm(x, w, b, eps, kind)
    xh = O.norm(x, None, None, eps, kind)[0]
    ww = np.ones(x.shape[1]) if w is None else w
    r = rstd[:, None]
    biggest = np.abs(x).max(axis=1, keepdims=True) if kind == "layer" else 0.0
    e_xh = K * U32 * (np.abs(xh) + r * biggest)
    pre = np.abs(ww) * e_xh + 4 * U32 * (np.abs(xh * ww) + (0 if b is None else np.abs(b)))
    res = [(y, u * np.abs(y) + pre + tiny(dtype))]
    if dy is None:
        return res
    dx, dw, db = O.norm_grad(dy, x, w, eps, kind)
    g = np.abs(dy * ww)
    mg, mgx = g.mean(1, keepdims=True), (g * np.abs(xh)).mean(1, keepdims=True)
    e = r * (K * U32 * (g + mg + np.abs(xh) * mgx) + e_xh * mgx
             + np.abs(xh) * (g * e_xh).mean(1, keepdims=True))
    e = e + K * U32 * r * (g + mg + np.abs(xh) * mgx)
    res.append((dx, u * np.abs(dx) + e + tiny(dtype)))
    uw = unit(wdtype)
    sums = 256 + x.shape[0] / 16        # longest chain of additions of one column
    res.append((dw, uw * np.abs(dw) + (np.abs(dy) * e_xh).sum(0)
                + sums * U32 * np.abs(dy * xh).sum(0) + tiny(wdtype)))
    res.append((db, uw * np.abs(db) + sums * U32 * np.abs(dy).sum(0) + tiny(wdtype)))
    return res


SHAPES = [(1, 1), (3, 7), (1, 7168), (5, 32), (33, 33), (600, 128), (601, 129), (37, 1003),
          (700, 250), (64, 2048), (593, 2048), (9, 4100), (21, 7168), (7, 8200), (5, 16384),
          (3, 16385), (4, 33000), (2, 70000), (1777, 96), (1300, 512), (1185, 1032),
          (5000, 64), (3001, 257), (4747, 33), (2600, 1024), (1200, 2056), (1190, 7168), (1184, 8200), (1500, 4096), (1184, 16384)]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"),
                                          ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm(rows, cols, dtype, wdtype, kind):
    g = gen(rows * 7 + cols)
    dt, wdt = DT[dtype], DT[wdtype]
    x = randn(g, rows, cols, dtype=dt, scale=1.5, shift=0.3)
    w = randn(g, cols, dtype=wdt, scale=0.2, shift=1.0)
    b = randn(g, cols, dtype=wdt, scale=0.2) if kind == "layer" else None
    dy = randn(g, rows, cols, dtype=dt, scale=0.5)
    y, mean, rstd = ops.norm_forward(x, w, b, eps=1e-5, kind=kind, save=True)
    dx, dw, db = ops.norm_backward(dy, x, w, mean, rstd, kind=kind, bias=b is not None)
    want = norm_bounds(f64(x), f64(w), None if b is None else f64(b), f64(dy), dt, wdt, kind, 1e-5)
    for name, got, (ref, tol) in zip(("y", "dx", "dweight", "dbias"), (y, dx, dw, db), want):
        if got is not None:
            close(got, ref, tol, name)
    # the same bits again, and the saved statistics change nothing
    assert torch.equal(y, ops.norm_forward(x, w, b, eps=1e-5, kind=kind))
    again = ops.norm_backward(dy, x, w, mean, rstd, kind=kind, bias=b is not None)
    for one, two in zip((dx, dw, db), again):
        assert one is None or torch.equal(one, two)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_without_parameters_and_partial_gradients(kind):
    g = gen(3)
    x, dy = randn(g, 50, 264), randn(g, 50, 264)
    y, mean, rstd = ops.norm_forward(x, kind=kind, save=True)
    want = norm_bounds(f64(x), None, None, f64(dy), torch.bfloat16, torch.bfloat16, kind, 1e-5)
    close(y, *want[0], "y")
    dx, dw, db = ops.norm_backward(dy, x, None, mean, rstd, kind=kind)
    assert dw is None and db is None
    close(dx, *want[1], "dx")
    w = randn(g, 264, shift=1.0)
    full = ops.norm_backward(dy, x, w, mean, rstd, kind=kind)
    only = ops.norm_backward(dy, x, w, mean, rstd, kind=kind, need_dx=False)
    assert only[0] is None and torch.equal(only[1], full[1])
    none = ops.norm_backward(dy, x, w, mean, rstd, kind=kind, need_dweight=False)
    assert none[1] is None and torch.equal(none[0], full[0])


def strided_variants(t):
    """The same values behind other strides and alignments."""
    rows, cols = t.shape
    wide = torch.zeros((rows, cols + 24), dtype=t.dtype, device=t.device)
    wide[:, 8:8 + cols] = t                       # 16-byte aligned rows
    odd = torch.zeros((rows, cols + 5), dtype=t.dtype, device=t.device)
    odd[:, 3:3 + cols] = t                        # rows at any element
    cm = t.t().contiguous().t()                   # column-major
    return {"padded": wide[:, 8:8 + cols], "odd": odd[:, 3:3 + cols], "column_major": cm}


@pytest.mark.parametrize("variant", ["padded", "odd", "column_major"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_strides(variant, dtype):
    g = gen(4)
    x, dy = randn(g, 65, 520, dtype=DT[dtype]), randn(g, 65, 520, dtype=DT[dtype])
    w = randn(g, 520, dtype=DT[dtype], shift=1.0)
    want = norm_bounds(f64(x), f64(w), None, f64(dy), DT[dtype], DT[dtype], "layer", 1e-5)
    xv, dyv = strided_variants(x)[variant], strided_variants(dy)[variant]
    y, mean, rstd = ops.norm_forward(xv, w, save=True)
    dx, dw, _ = ops.norm_backward(dyv, xv, w, mean, rstd)
    for name, got, (ref, tol) in zip(("y", "dx", "dweight"), (y, dx, dw), want):
        close(got, ref, tol, name)
    # a weight that starts at an odd element
    w2 = torch.cat([w[:1], w])[1:]
    close(ops.norm_forward(x, w2), *want[0], "y with an odd weight")


@pytest.mark.parametrize("variant", ["padded", "odd"])
@pytest.mark.parametrize("cols", [40, 300, 1000])
def test_norm_strides_many_rows(variant, cols):
    g = gen(14 + cols)
    x, dy = randn(g, 700, cols), randn(g, 700, cols)
    w = randn(g, cols, shift=1.0)
    want = norm_bounds(f64(x), f64(w), None, f64(dy), torch.bfloat16, torch.bfloat16, "layer", 1e-5)
    xv, dyv = strided_variants(x)[variant], strided_variants(dy)[variant]
    y, mean, rstd = ops.norm_forward(xv, w, save=True)
    dx, dw, _ = ops.norm_backward(dyv, xv, w, mean, rstd)
    for name, got, (ref, tol) in zip(("y", "dx", "dweight"), (y, dx, dw), want):
        close(got, ref, tol, name)


def test_norm_at_the_end_of_an_odd_matrix():
    # the last bytes of a contiguous matrix whose size is no multiple of 16 bytes: nothing
    # behind it is read into the result, nothing behind the output is written
    rows, cols = 1201, 333
    g = gen(15)
    buf = torch.full((rows * cols + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = buf[:rows * cols].view(rows, cols)
    x.copy_(randn(g, rows, cols))
    out = torch.full((rows * cols + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    lib = load_library()
    assert lib.moe_norm_forward(0, 0, 0, rows, cols, x.data_ptr(), cols, None, None, 1e-5,
                                out.data_ptr(), cols, None, None,
                                torch.cuda.current_stream().cuda_stream) == 0
    want = norm_bounds(f64(x), None, None, None, torch.bfloat16, torch.bfloat16, "layer", 1e-5)
    close(out[:rows * cols].view(rows, cols), *want[0], "y")
    assert torch.equal(out[rows * cols:], torch.full_like(out[rows * cols:], 7.0))


def test_norm_in_place():
    # y over x, and dx over dy, as the C interface allows
    lib = load_library()
    stream = torch.cuda.current_stream().cuda_stream
    for rows, cols in ((5, 520), (700, 520), (700, 333), (3, 70000)):
        g = gen(16)
        x, dy = randn(g, rows, cols), randn(g, rows, cols)
        y, mean, rstd = ops.norm_forward(x, save=True)
        dx = ops.norm_backward(dy, x, None, mean, rstd)[0]
        x2, dy2 = x.clone(), dy.clone()
        assert lib.moe_norm_backward(0, 0, 0, rows, cols, dy2.data_ptr(), cols, x.data_ptr(), cols,
                                     None, mean.data_ptr(), rstd.data_ptr(), dy2.data_ptr(), cols,
                                     None, None, None, 0, stream) == 0
        assert lib.moe_norm_forward(0, 0, 0, rows, cols, x2.data_ptr(), cols, None, None, 1e-5,
                                    x2.data_ptr(), cols, None, None, stream) == 0
        assert torch.equal(x2, y) and torch.equal(dy2, dx)


def test_norm_broadcast_gradient_and_leading_dimensions():
    g = gen(5)
    x = randn(g, 3, 4, 72, dtype=torch.float32)
    dy = randn(g, 72, dtype=torch.float32).expand(3, 4, 72)
    w = randn(g, 72, dtype=torch.float32)
    x.requires_grad_(True)
    w.requires_grad_(True)
    ops.layer_norm(x, w).backward(dy)
    want = norm_bounds(f64(x).reshape(12, 72), f64(w), None, f64(dy).reshape(12, 72),
                       torch.float32, torch.float32, "layer", 1e-5)
    close(x.grad.reshape(12, 72), *want[1], "dx")
    close(w.grad, *want[2], "dweight")


def test_norm_far_from_zero_and_extreme_rows():
    g = gen(6)
    x = randn(g, 40, 1000, dtype=torch.float32, shift=1000.0)
    want = norm_bounds(f64(x), None, None, None, torch.float32, torch.float32, "layer", 1e-5)
    close(ops.norm_forward(x), *want[0], "far from zero")
    # a constant row has no variance: y = bias; a zero row under RMS: 0
    c = torch.full((2, 1000), 3.0, device="cuda")
    assert torch.equal(ops.norm_forward(c), torch.zeros_like(c))
    z = torch.zeros((2, 1000), device="cuda", dtype=torch.bfloat16)
    assert torch.equal(ops.norm_forward(z, kind="rms"), z)
    # a row with NaN or an infinity stays alone
    y0 = ops.norm_forward(x)
    x2 = x.clone()
    x2[3, 7], x2[5, 1] = float("nan"), float("inf")
    y1 = ops.norm_forward(x2)
    keep = [i for i in range(40) if i not in (3, 5)]
    assert torch.equal(y0[keep], y1[keep])
    assert torch.isnan(y1[3]).all() and not torch.isfinite(y1[5, 1])


def test_norm_empty_batch():
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    b = torch.ones(64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = ops.layer_norm(x, w, b)
    assert y.shape == (0, 64)
    y.sum().backward()
    assert torch.equal(w.grad, torch.zeros_like(w)) and torch.equal(b.grad, torch.zeros_like(b))


# ------------------------------------------------------------------------ dropout
def drop_tol(x, res, p, dtype, want):
    s = 1 / (1 - p)
    return unit(dtype) * np.abs(want) + 4 * U32 * (np.abs(x) * s + (0 if res is None else
                                                                    np.abs(res))) + tiny(dtype)


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 3), (1, 8), (3, 7), (128, 2048), (777, 1001),
                                       (1, 100003)])
def test_dropout_add(rows, cols, dtype, p):
    g = gen(rows + cols)
    dt = DT[dtype]
    x, res = randn(g, rows, cols, dtype=dt), randn(g, rows, cols, dtype=dt)
    seed, offset = -3 - cols, 2 ** 40 + rows       # a negative seed: its 64 bits count
    rng = torch.tensor([seed, offset], device="cuda")
    out = ops.dropout_add_forward(x, res, p, rng)
    want = O.dropout_add(f64(x), f64(res), p, seed, offset)
    close(out, want, drop_tol(f64(x), f64(res), p, dt, want), "out")
    dx = ops.dropout_add_backward(x, p, rng)
    want = O.dropout_add(f64(x), None, p, seed, offset)
    close(dx, want, drop_tol(f64(x), None, p, dt, want), "dx")
    keep = O.dropout_keep(rows * cols, p, seed, offset).reshape(rows, cols)
    assert ((f64(dx) != 0) <= keep).all()          # dropped: exactly zero


@pytest.mark.parametrize("variant", ["padded", "odd", "column_major"])
def test_dropout_strides(variant):
    g = gen(8)
    x, res = randn(g, 33, 130), randn(g, 33, 130)
    rng = torch.tensor([11, 12], device="cuda")
    want = ops.dropout_add_forward(x, res, 0.3, rng)
    xv, rv = strided_variants(x)[variant], strided_variants(res)[variant]
    for a, b in ((xv, res), (x, rv), (xv, rv)):
        assert torch.equal(ops.dropout_add_forward(a, b, 0.3, rng), want)


def test_dropout_masks_non_finite_and_drops_all():
    n = 4096
    rng = torch.tensor([1, 2], device="cuda")
    x = torch.full((1, n), float("nan"), device="cuda")
    x[:, ::2] = float("inf")
    res = torch.ones_like(x)
    out = ops.dropout_add_forward(x, res, 0.5, rng)
    keep = torch.from_numpy(O.dropout_keep(n, 0.5, 1, 2)).cuda().reshape(1, n)
    assert torch.equal(out[~keep], torch.ones_like(out[~keep]))
    assert not torch.isfinite(out[keep]).any()
    assert torch.equal(ops.dropout_add_forward(x, res, 1.0, rng), res)
    assert torch.equal(ops.dropout_add_forward(x, res, 1.0 - 1e-12, rng), res)


def test_dropout_beyond_32_bits():
    # more elements than one launch covers: the mask's counter goes on across them
    n = (1 << 34) + (1 << 33) + 4099
    rng = torch.tensor([7, 8], device="cuda")
    x = torch.ones((1, n), dtype=torch.bfloat16, device="cuda")
    out = ops.dropout_add_forward(x, None, 0.5, rng)
    for first in (0, (1 << 33) - 4096, (1 << 34) - 4096, 3 * (1 << 33) - 4096, n - 8195):
        m = min(8192, n - first)
        keep = torch.from_numpy(O.dropout_keep(m, 0.5, 7, 8, first)).cuda()
        assert torch.equal(out[0, first:first + m], torch.where(keep, 2.0, 0.0).bfloat16())


def test_dropout_gradients_and_changed_rng():
    g = gen(9)
    x = randn(g, 40, 96, dtype=torch.float32).requires_grad_(True)
    res = randn(g, 40, 96, dtype=torch.float32).requires_grad_(True)
    rng = torch.tensor([5, 6], device="cuda")
    dout = randn(g, 40, 96, dtype=torch.float32)
    ops.dropout_add(x, res, 0.4, rng).backward(dout)
    want = O.dropout_add(f64(dout), None, 0.4, 5, 6)
    close(x.grad, want, drop_tol(f64(dout), None, 0.4, torch.float32, want), "dx")
    assert torch.equal(res.grad, dout)
    out = ops.dropout_add(x, res, 0.4, rng)
    rng[1] += 1
    with pytest.raises(RuntimeError):              # the mask could not be drawn again
        out.sum().backward()


def test_dropout_graph_draws_anew_when_rng_changes():
    g = gen(10)
    x, res = randn(g, 64, 128), randn(g, 64, 128)
    rng = torch.tensor([3, 0], device="cuda")
    ops.dropout_add_forward(x, res, 0.2, rng)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.dropout_add_forward(x, res, 0.2, rng)
        rng[1] += 1
    for step in range(3):
        graph.replay()
        want = ops.dropout_add_forward(x, res, 0.2, torch.tensor([3, step], device="cuda"))
        assert torch.equal(out, want)


# ------------------------------------------------------------------------ gated feed-forward
def ffn_case(T, d, f, dtype, seed=0):
    g = gen(seed * 1000 + T + d + f)
    dt = DT[dtype]
    return (randn(g, T, d, dtype=dt), randn(g, f, d, dtype=dt, scale=d ** -0.5),
            randn(g, f, d, dtype=dt, scale=d ** -0.5), randn(g, d, f, dtype=dt, scale=f ** -0.5),
            randn(g, T, d, dtype=dt, scale=0.25))


def ffn_bounds(x, W1, W3, W2, dout, act, dtype):
    """{name: (value, tolerance)} of out, dx, dW1, dW3, dW2.

    A tensor-core reduction of n products may truncate each of its additions: it is off by
    at most (n / 8 + 16) * 2^-23 times the sum of magnitudes (chains of at least 8 products
    a step). act, act' and act'' of SiLU and GELU are at most |a|, 1.13 and 1 in size; the
    fast exponential is good to 2 + 1.18 |z| units, below 2^-18 for |z| < 20."""
    u, t = unit(dtype), tiny(dtype)
    red = lambda n: (n / 8 + 16) * 2.0 ** -23            # noqa: E731
    A = np.abs
    T, d = x.shape
    f = W1.shape[0]
    fast = 2.0 ** -17
    out, gate, up = O.gated_ffn(x, W1, W3, W2, act)
    val, der = O.activation(gate, act)
    e_g, e_u = red(d) * (A(x) @ A(W1).T), red(d) * (A(x) @ A(W3).T)
    h = val * up
    e_h = u * A(h) + 1.13 * e_g * A(up) + A(val) * e_u + fast * A(h) + t
    res = {"out": (out, u * A(out) + (e_h + red(f) * A(h)) @ A(W2).T + t)}
    dx, dW1, dW3, dW2 = O.gated_ffn_grad(dout, x, W1, W3, W2, act)
    e_g, e_u = e_g + u * A(gate) + t, e_u + u * A(up) + t
    dh = dout @ W2
    e_dh = red(d) * (A(dout) @ A(W2))
    dg, du = dh * up * der, dh * val
    e_dg = u * A(dg) + e_dh * A(up * der) + A(dh) * (e_u * A(der) + A(up) * e_g) \
        + fast * A(dh * up) + t
    e_du = u * A(du) + e_dh * A(val) + A(dh) * 1.13 * e_g + fast * A(dh) * (A(val) + 1) + t
    e_h = u * A(h) + 1.13 * e_g * A(up) + A(val) * e_u + fast * A(h) + t
    res["dx"] = (dx, u * A(dx) + (e_dg + red(2 * f) * A(dg)) @ A(W1)
                 + (e_du + red(2 * f) * A(du)) @ A(W3) + t)
    res["dW1"] = (dW1, u * A(dW1) + (e_dg + red(T) * A(dg)).T @ A(x) + t)
    res["dW3"] = (dW3, u * A(dW3) + (e_du + red(T) * A(du)).T @ A(x) + t)
    res["dW2"] = (dW2, u * A(dW2) + A(dout).T @ (e_h + red(T) * A(h)) + t)
    # products of two of these errors
    return {k: (v, 1.05 * tol) for k, (v, tol) in res.items()}


def check_ffn(T, d, f, dtype, act, seed=0):
    x, W1, W3, W2, dout = ffn_case(T, d, f, dtype, seed)
    out, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, act, save=True)
    grads = ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up, act)
    ops.device_status()
    want = ffn_bounds(*(f64(t) for t in (x, W1, W3, W2, dout)), act, DT[dtype])
    for name, got in zip(("out", "dx", "dW1", "dW3", "dW2"), (out, *grads)):
        ref, tol = want[name]
        close(got, ref, tol, name)
        # at most six independent roundings in a row, each u / sqrt(3) in the mean square:
        # sqrt(2) u; doubled for sums whose terms do not average out. Values near fp16's
        # smallest count absolutely.
        off, size = np.linalg.norm(f64(got) - ref), np.linalg.norm(ref)
        assert off <= 3 * unit(DT[dtype]) * size + tiny(DT[dtype]) * math.sqrt(ref.size), \
            f"{name}: relative error {off / size}"
    # without saved pre-activations: the same bits
    assert torch.equal(out, ops.gated_ffn_forward(x, W1, W3, W2, act))


@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("fp16", "gelu")])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("d,f", [(8, 8), (64, 64), (72, 40), (136, 264)])
def test_gated_ffn_small(T, d, f, dtype, act):
    check_ffn(T, d, f, dtype, act)


@pytest.mark.parametrize("T,d,f,dtype,act", [
    (1, 2048, 1408, "bf16", "gelu"), (24, 2048, 2816, "fp16", "silu"),
    (333, 2048, 1408, "fp16", "gelu"), (333, 2048, 1408, "bf16", "silu"),
    (5, 1000, 5000, "bf16", "silu"), (130, 4104, 520, "bf16", "silu"),
    (1000, 520, 1032, "bf16", "gelu"), (40, 8, 2048, "fp16", "silu"),
    (3, 7168, 8, "bf16", "silu"),
])
def test_gated_ffn_larger(T, d, f, dtype, act):
    check_ffn(T, d, f, dtype, act)


@pytest.mark.parametrize("T,d,f,dtype,act", [
    # enough tiles for the CTA-pair kernel in every product; ragged in every dimension
    (2321, 2088, 2632, "bf16", "silu"), (2560, 2048, 2560, "fp16", "gelu"),
])
def test_gated_ffn_pairs(T, d, f, dtype, act):
    check_ffn(T, d, f, dtype, act)


@pytest.mark.parametrize("T,d,f", [(129, 136, 264), (2321, 2088, 2632)])
def test_gated_ffn_repeats_bit_for_bit_and_subsets(T, d, f):
    x, W1, W3, W2, dout = ffn_case(T, d, f, "bf16", 1)
    out, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, save=True)
    full = ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up)
    for _ in range(3):
        assert torch.equal(out, ops.gated_ffn_forward(x, W1, W3, W2))
        again = ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up)
        assert all(torch.equal(a, b) for a, b in zip(full, again))
    for needs in ((True, False, False, False), (False, True, False, True),
                  (False, False, True, False), (False, False, False, True)):
        part = ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up, needs=needs)
        for want, got, need in zip(full, part, needs):
            assert (got is None) != need and (got is None or torch.equal(got, want))


def test_gated_ffn_strides_and_leading_dimensions():
    x, W1, W3, W2, dout = ffn_case(65, 136, 264, "bf16", 2)
    out, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, save=True)
    full = ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up)
    xs, ds = strided_variants(x), strided_variants(dout)
    for v in xs:
        assert torch.equal(ops.gated_ffn_forward(xs[v], W1, W3, W2), out)
        got = ops.gated_ffn_backward(ds[v], xs[v], W1, W3, W2, gate, up)
        assert all(torch.equal(a, b) for a, b in zip(full, got))
    assert torch.equal(ops.gated_ffn_forward(x.view(5, 13, 136), W1, W3, W2), out.view(5, 13, 136))


def test_gated_ffn_rows_do_not_mix():
    # a NaN token reaches its own output and x gradient, and no other token's
    x, W1, W3, W2, dout = ffn_case(140, 136, 264, "bf16", 3)
    out, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, save=True)
    x2 = x.clone()
    x2[77] = float("nan")
    out2, gate2, up2 = ops.gated_ffn_forward(x2, W1, W3, W2, save=True)
    keep = [i for i in range(140) if i != 77]
    assert torch.equal(out[keep], out2[keep]) and torch.isnan(out2[77]).all()
    dx = ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up)[0]
    dx2 = ops.gated_ffn_backward(dout, x2, W1, W3, W2, gate2, up2)[0]
    assert torch.equal(dx[keep], dx2[keep])


def test_gated_ffn_large_pre_activations():
    # gates far out on both sides: SiLU and GELU saturate without NaN
    x = torch.full((4, 64), 8.0, device="cuda", dtype=torch.bfloat16)
    x[2:] = -8.0
    W1 = torch.full((64, 64), 8.0, device="cuda", dtype=torch.bfloat16)
    W3 = torch.full((64, 64), 0.125, device="cuda", dtype=torch.bfloat16)
    W2 = torch.full((64, 64), 2.0 ** -12, device="cuda", dtype=torch.bfloat16)
    for act in ("silu", "gelu"):
        out, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, act, save=True)
        assert torch.equal(gate[:2], torch.full_like(gate[:2], 4096.0))
        assert torch.equal(out[:2], torch.full_like(out[:2], 4096.0))   # 64 * 4096 * 64 * 2^-12
        assert torch.equal(out[2:], torch.zeros_like(out[2:]))
        for gr in ops.gated_ffn_backward(x, x, W1, W3, W2, gate, up, act):
            assert torch.isfinite(gr).all()


def test_gated_ffn_empty_batch():
    _, W1, W3, W2, _ = ffn_case(1, 64, 72, "bf16", 4)
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    out, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, save=True)
    assert out.shape == (0, 64)
    grads = ops.gated_ffn_backward(x, x, W1, W3, W2, gate, up)
    assert all(torch.equal(gr, torch.zeros_like(gr)) for gr in grads)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_ffn_gradient_against_differences(act):
    # along a random direction v: (L(w + hv) - L(w - hv)) / 2h of the fp64 forward, where
    # L = sum(out * dout); the third-order term is below 1e-6 relative here, so the
    # difference is the kernels' own error: the bound of each gradient, summed against |v|
    x, W1, W3, W2, dout = ffn_case(70, 72, 136, "bf16", 5)
    _, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, act, save=True)
    grads = ops.gated_ffn_backward(dout, x, W1, W3, W2, gate, up, act)
    at = [f64(t) for t in (x, W1, W3, W2)]
    bounds = ffn_bounds(*at, f64(dout), act, torch.bfloat16)
    rng = np.random.default_rng(0)
    h = 1e-5
    for i, (name, got) in enumerate(zip(("dx", "dW1", "dW3", "dW2"), grads)):
        v = rng.normal(size=at[i].shape)
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + h * v, at[i] - h * v
        diff = ((O.gated_ffn(*hi, act)[0] - O.gated_ffn(*lo, act)[0]) * f64(dout)).sum() / (2 * h)
        tol = (bounds[name][1] * np.abs(v)).sum() + 1e-5 * abs(diff)
        assert abs(diff - (f64(got) * v).sum()) <= tol, name


def test_refusals_on_the_gpu():
    x, W1, W3, W2, dout = ffn_case(4, 64, 72, "bf16", 6)
    out, gate, up = ops.gated_ffn_forward(x, W1, W3, W2, save=True)
    y, mean, rstd = ops.norm_forward(x, save=True)
    rng = torch.tensor([1, 2], device="cuda")
    bad = [
        lambda: ops.gated_ffn_forward(x.float(), W1.float(), W3.float(), W2.float()),
        lambda: ops.gated_ffn_forward(x, W1.t(), W3, W2),
        lambda: ops.gated_ffn_forward(x, W1, W3.half(), W2),
        lambda: ops.gated_ffn_forward(x[:, :60].contiguous(), W1[:, :60].contiguous(),
                                      W3[:, :60].contiguous(), W2[:60].contiguous()),
        lambda: ops.gated_ffn_forward(x, W1, W3, W2, "tanh"),
        lambda: ops.gated_ffn_forward(x, W1, W3, W2.cpu()),
        lambda: ops.gated_ffn_backward(dout[:2], x, W1, W3, W2, gate, up),
        lambda: ops.gated_ffn_backward(dout, x, W1, W3, W2, gate[:2], up),
        lambda: ops.norm_forward(x, kind="batch"),
        lambda: ops.norm_forward(x, torch.ones(63, device="cuda")),
        lambda: ops.norm_forward(x, torch.ones(64, device="cuda", dtype=torch.float16)),
        lambda: ops.norm_forward(x, None, torch.ones(64, device="cuda"), kind="rms"),
        lambda: ops.norm_forward(x, eps=-1.0),
        lambda: ops.norm_forward(x.double()),
        lambda: ops.norm_backward(dout, x, None, mean[:2], rstd),
        lambda: ops.norm_backward(dout, x, None, None, rstd),
        lambda: ops.dropout_add_forward(x, dout[:2], 0.1, rng),
        lambda: ops.dropout_add_forward(x, dout, 1.5, rng),
        lambda: ops.dropout_add_forward(x, dout, 0.1, None),
        lambda: ops.dropout_add_forward(x, dout, 0.1, rng.cpu()),
        lambda: ops.dropout_add_forward(x, dout, 0.1, rng.int()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(MoEError):
            call()
            pytest.fail(f"call {i} was not refused")


# ------------------------------------------------------------------------ together
def test_block_trains_like_the_formula():
    """x + dropout(ffn(norm(x))) through autograd against the oracle's chain rule. Its
    intermediate tensors (norm output, block output and their gradients) are rounded to
    bf16 between the operators, so the comparison is in the mean square: at most 10
    roundings in a row, 10 u."""
    T, d, f, p = 77, 136, 264, 0.25
    x, W1, W3, W2, dout = ffn_case(T, d, f, "bf16", 7)
    nw, nb = randn(gen(1), d, scale=0.1, shift=1.0), randn(gen(2), d, scale=0.1)
    rng = torch.tensor([21, 22], device="cuda")
    leaves = [t.requires_grad_(True) for t in (x, W1, W3, W2, nw, nb)]
    out = ops.gated_ffn_block(x, W1, W3, W2, nw, nb, norm="layer", activation="gelu", p=p, rng=rng)
    out.backward(dout)
    ax, a1, a3, a2, anw, anb = (f64(t) for t in leaves)
    h = O.norm(ax, anw, anb, 1e-5)[0]
    want_out = O.dropout_add(O.gated_ffn(h, a1, a3, a2, "gelu")[0], ax, p, 21, 22)
    dmid = O.dropout_add(f64(dout), None, p, 21, 22)
    dh, d1, d3, d2 = O.gated_ffn_grad(dmid, h, a1, a3, a2, "gelu")
    dxn, dnw, dnb = O.norm_grad(dh, ax, anw)
    want = (want_out, dxn + f64(dout), d1, d3, d2, dnw, dnb)
    for name, got, ref in zip(("out", "x", "W1", "W3", "W2", "weight", "bias"),
                              (out, *(t.grad for t in leaves)), want):
        off = np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)
        assert off <= 10 * unit(torch.bfloat16), f"{name}: {off}"


def test_moe_layer_block():
    from mixture_experts_ffn_expert_b200.inputs import WORKLOADS, make_layer_inputs
    from mixture_experts_ffn_expert_b200.layer import MoELayer
    s = WORKLOADS["tiny_t256_d128_f64_e31k7_s1"]
    inp = make_layer_inputs(s, seed=0, device="cuda")
    layer = MoELayer(s.d, s.f, s.n_routed, s.top_k, s.n_shared, s.renorm, inp, bias=inp["bias"])
    w = randn(gen(3), s.d, scale=0.1, shift=1.0)
    x = inp["x"]
    rng = torch.tensor([1, 2], device="cuda")
    mid = layer(ops.norm_forward(x, w, kind="rms"))
    assert torch.equal(layer.block(x, w), ops.dropout_add_forward(mid, x, 0.0, None))
    want = O.dropout_add(f64(mid), f64(x), 0.0, 0, 0)
    close(layer.block(x, w), want, drop_tol(f64(mid), f64(x), 0.0, torch.bfloat16, want), "block")
    assert torch.equal(layer.block(x, w, p=0.1, rng=rng),
                       ops.dropout_add_forward(mid, x, 0.1, rng))


def test_training_step_in_a_graph_and_on_other_streams():
    T, d, f = 200, 136, 264
    x, W1, W3, W2, dout = ffn_case(T, d, f, "bf16", 8)
    nw = randn(gen(4), d, scale=0.1, shift=1.0)
    rng = torch.tensor([4, 5], device="cuda")

    def step():
        h, mean, rstd = ops.norm_forward(x, nw, save=True)
        y, gate, up = ops.gated_ffn_forward(h, W1, W3, W2, save=True)
        out = ops.dropout_add_forward(y, x, 0.1, rng)
        dy = ops.dropout_add_backward(dout, 0.1, rng)
        dh, d1, d3, d2 = ops.gated_ffn_backward(dy, h, W1, W3, W2, gate, up)
        dx, dnw, _ = ops.norm_backward(dh, x, nw, mean, rstd)
        return out, dx, d1, d3, d2, dnw

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    results = []
    for s in streams:                       # at the same time on three streams
        with torch.cuda.stream(s):
            results.append(step())
    torch.cuda.synchronize()
    for r in results:
        assert all(torch.equal(a, b) for a, b in zip(want, r))
    graphs = []
    for _ in range(2):                      # two captured steps replayed against each other
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step()
        graphs.append((graph, res))
    new = randn(gen(5), T, d)
    old = x.clone()
    for source in (new, old):
        x.copy_(source)
        ref = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for i, (graph, _) in enumerate(graphs):
            with torch.cuda.stream(streams[i]):
                graph.replay()
        torch.cuda.synchronize()
        for _, res in graphs:
            assert all(torch.equal(a, b) for a, b in zip(ref, res))
    assert all(torch.equal(a, b) for a, b in zip(want, ref))
    load_library()
    ops.device_status()


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    """Seeded shapes over the whole range of each operator (sizes log-uniform, odd ones
    among them), with the bounds of the fixed cases."""
    import random
    r = random.Random(seed)
    log = lambda lo, hi: int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    d, f = 8 * log(1, 160), 8 * log(1, 160)
    check_ffn(log(1, 1500), d, f, r.choice(["bf16", "fp16"]), r.choice(["silu", "gelu"]), seed)
    for _ in range(3):
        cols = log(1, 12000)
        rows = log(1, max(1, min(4000, 3_000_000 // cols)))
        test_norm(rows, cols, *r.choice([("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"),
                                         ("fp32", "fp32")]), r.choice(["layer", "rms"]))
        test_dropout_add(rows, cols, r.choice(["bf16", "fp16", "fp32"]),
                         r.choice([0.0, 0.1, 0.37, 0.9]))


FIRST_CALL = """
import torch
from mixture_experts_ffn_expert_b200 import ops
g = lambda *s: torch.randn(*s, device="cuda").bfloat16()
x, W1, W3, W2 = g(40, 64), g(72, 64), g(72, 64), g(64, 72)
rng = torch.tensor([1, 2], device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    h = ops.norm_forward(x, kind="rms")
    y, gate, up = ops.gated_ffn_forward(h, W1, W3, W2, save=True)
    grads = ops.gated_ffn_backward(y, h, W1, W3, W2, gate, up)
    out = ops.dropout_add_forward(y, x, 0.1, rng)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, ops.dropout_add_forward(
    ops.gated_ffn_forward(ops.norm_forward(x, kind="rms"), W1, W3, W2), x, 0.1, rng))
ops.device_status()
print("captured")
"""


def test_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_many_host_threads_and_streams():
    # eight host threads, each on its own stream with its own inputs, at the same time
    import threading
    cases = [ffn_case(T, 136, 264, "bf16", 20 + i)
             for i, T in enumerate((1, 7, 33, 64, 129, 200, 300, 500))]

    def step(c):
        x, W1, W3, W2, dout = c
        h, mean, rstd = ops.norm_forward(x, save=True)
        y, gate, up = ops.gated_ffn_forward(h, W1, W3, W2, save=True)
        grads = ops.gated_ffn_backward(dout, h, W1, W3, W2, gate, up)
        return (y, *grads, ops.norm_backward(grads[0], x, None, mean, rstd)[0])

    want = [step(c) for c in cases]
    torch.cuda.synchronize()
    got, errors = [None] * len(cases), []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[i] = step(cases[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:     # reported by the test's thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_same_tensor_twice():
    # one tensor as several arguments: W1 as W3, x as residual and as the gradient
    x, W1, _, W2, _ = ffn_case(50, 136, 264, "bf16", 30)
    out, gate, up = ops.gated_ffn_forward(x, W1, W1, W2, save=True)
    assert torch.equal(gate, up)
    dx, d1, d3, d2 = ops.gated_ffn_backward(x, x, W1, W1, W2, gate, up)
    want = ffn_bounds(*(f64(t) for t in (x, W1, W1, W2, x)), "silu", torch.bfloat16)
    for name, got in zip(("out", "dx", "dW1", "dW3", "dW2"), (out, dx, d1, d3, d2)):
        close(got, *want[name], name)
    rng = torch.tensor([3, 4], device="cuda")
    got = ops.dropout_add_forward(x, x, 0.25, rng)
    want = O.dropout_add(f64(x), f64(x), 0.25, 3, 4)
    close(got, want, drop_tol(f64(x), f64(x), 0.25, torch.bfloat16, want), "x twice")


def test_no_grad_saves_nothing():
    # leaves that want gradients under no_grad: the forward's bits, and no pre-activations
    T, d, f = 520, 136, 4096
    x, W1, W3, W2, _ = ffn_case(T, d, f, "bf16", 31)
    rng = torch.tensor([5, 6], device="cuda")
    want = ops.gated_ffn_forward(x, W1, W3, W2)
    norm = ops.norm_forward(x, kind="rms")
    drop = ops.dropout_add_forward(want, x, 0.25, rng)
    block = ops.gated_ffn_block(x, W1, W3, W2, p=0.25, rng=rng)
    for t in (x, W1, W3, W2):
        t.requires_grad_(True)
    with torch.no_grad():
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        out = ops.gated_ffn(x, W1, W3, W2)
        peak = torch.cuda.max_memory_allocated() - before
        assert torch.equal(ops.rms_norm(x), norm)
        assert torch.equal(ops.dropout_add(out, x, 0.25, rng), drop)
        again = ops.gated_ffn_block(x, W1, W3, W2, p=0.25, rng=rng)
    assert torch.equal(out, want) and not out.requires_grad
    assert torch.equal(again, block) and not again.requires_grad
    # act(gate) * up (T, f) and the output; gate and up would be two more of the first
    assert peak < 2 * (T * f * 2)


def test_negated_views_are_refused_or_resolved():
    # a view with torch's negative bit holds the unnegated values in memory
    x = randn(gen(32), 6, 64, dtype=torch.float32)
    neg = torch._neg_view(x)
    rng = torch.tensor([5, 6], device="cuda")
    for call in (lambda: ops.norm_forward(neg), lambda: ops.dropout_add_forward(neg, x, 0.5, rng),
                 lambda: ops.dropout_add_forward(x, neg, 0.5, rng)):
        with pytest.raises(MoEError):
            call()
    assert torch.equal(ops.norm_forward(neg.resolve_neg()), ops.norm_forward(-x))
