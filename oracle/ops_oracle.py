"""fp64 oracle of the operators around the layer: norm, gated feed-forward block, dropout.

Plain NumPy definitions, written from the formulas; nothing is imported from the package.

* layer norm: xh = (x - mean) / sqrt(var + eps), var the mean squared difference from the
  mean; RMS norm: xh = x / sqrt(mean(x^2) + eps); y = xh * weight + bias. Gradients by the
  chain rule through mean and variance.
* gated block: out = (act(x W1^T) * (x W3^T)) W2^T, act SiLU or GELU in its tanh form.
* dropout: element e (row-major) is kept when word e % 4 of Philox-4x32-10 at counter
  (low 64 bits e // 4, high 64 bits offset) and key seed is >= round(p * 2^32). The
  generator is written from Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
  easy as 1, 2, 3" (SC 2011).
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------------ norm
def norm(x, weight=None, bias=None, eps=1e-5, kind="layer"):
    """y, mean, rstd of the rows of x (rows, cols)."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1) if kind == "layer" else np.zeros(x.shape[0])
    var = ((x - mean[:, None]) ** 2).mean(axis=1)
    rstd = 1.0 / np.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    return y, mean, rstd


def norm_grad(dy, x, weight=None, eps=1e-5, kind="layer"):
    """dx, dweight, dbias."""
    dy = np.asarray(dy, dtype=np.float64)
    x = np.asarray(x, dtype=np.float64)
    xh, _, rstd = norm(x, None, None, eps, kind)
    n = x.shape[1]
    g = dy if weight is None else dy * np.asarray(weight, dtype=np.float64)
    # d rstd / d x_j = -rstd^2 * xh_j / n, so each xh_i also moves by -xh_i xh_j rstd / n
    dx = g * rstd[:, None] - xh * rstd[:, None] * (g * xh).sum(axis=1, keepdims=True) / n
    if kind == "layer":
        dx = dx - rstd[:, None] * g.sum(axis=1, keepdims=True) / n
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


# ------------------------------------------------------------------------ gated block
def activation(a, name):
    """act(a) and act'(a)."""
    if name == "silu":
        e = np.exp(-np.abs(a))
        s = np.where(a >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
        return a * s, s + a * s * (1.0 - s)
    c = np.sqrt(2.0 / np.pi)
    t = np.tanh(c * (a + 0.044715 * a ** 3))
    return (0.5 * a * (1.0 + t),
            0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * a * a))


def gated_ffn(x, W1, W3, W2, act="silu"):
    """out, gate, up."""
    gate, up = x @ W1.T, x @ W3.T
    return (activation(gate, act)[0] * up) @ W2.T, gate, up


def gated_ffn_grad(dout, x, W1, W3, W2, act="silu"):
    """dx, dW1, dW3, dW2."""
    _, gate, up = gated_ffn(x, W1, W3, W2, act)
    val, der = activation(gate, act)
    dh = dout @ W2
    dgate, dup = dh * up * der, dh * val
    return dgate @ W1 + dup @ W3, dgate.T @ x, dup.T @ x, dout.T @ (val * up)


# ------------------------------------------------------------------------ dropout
def philox_4x32_10(counter, key):
    """counter: four uint32 arrays (or numbers), key: two numbers; four uint32 arrays."""
    mask = np.uint64(0xFFFFFFFF)
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(key[0]), int(key[1])]
    for _ in range(10):
        a = c[0] * np.uint64(0xD2511F53)       # 32 x 32 bits: no overflow of 64
        b = c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & mask,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return [np.asarray(v, dtype=np.uint32) for v in c]


def dropout_keep(n, p, seed, offset, first=0):
    """Truth value of each of the n elements from `first` (a multiple of 4) on: kept."""
    seed, offset = int(seed) & (2 ** 64 - 1), int(offset) & (2 ** 64 - 1)
    block = np.arange((n + 3) // 4, dtype=np.uint64) + np.uint64(first // 4)
    zero = np.zeros_like(block)
    words = philox_4x32_10(
        [block & np.uint64(0xFFFFFFFF), block >> np.uint64(32),
         zero + np.uint64(offset & 0xFFFFFFFF), zero + np.uint64(offset >> 32)],
        [seed & 0xFFFFFFFF, seed >> 32])
    w = np.stack(words, axis=1).reshape(-1)[:n].astype(np.uint64)
    return w >= np.uint64(round(p * 2 ** 32))


def dropout_add(x, residual, p, seed, offset):
    x = np.asarray(x, dtype=np.float64)
    keep = dropout_keep(x.size, p, seed, offset).reshape(x.shape)
    scaled = x / (1.0 - p) if p < 1 else np.zeros_like(x)
    out = np.where(keep, scaled, 0.0)
    return out if residual is None else out + np.asarray(residual, dtype=np.float64)
