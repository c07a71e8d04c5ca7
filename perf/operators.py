"""Measured cases of the training operators around the feed-forward layer.

Three operators, each in its plain form and through the package's entry points:

* ``ffn``: the gated feed-forward block ``out = (act(x W1^T) * (x W3^T)) W2^T`` (the
  shared expert of the layer, or a dense feed-forward layer), forward, and a training
  step (forward and backward: the gradients of x, W1, W3 and W2);
* ``norm``: layer norm and RMS norm over the rows of a token batch, forward, and
  forward with backward (the gradients of x, of the weight and of the bias);
* ``dropout``: ``out = residual + dropout(x)``, the mask from the counter-based
  generator Philox-4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2,
  3", 2011), never stored: the backward pass draws it again.

``run`` computes the plain form in fp32 with elementary torch operations, or, where
``own`` is true, calls the package. ``exact`` is the definition in fp64.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
LARGEST_FLOPS = 18 * 4096 * 4096 * 14336      # the largest listed training step
LARGEST_ELEMS = 8192 * 7168                   # the largest listed row batch


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token through the 14336-wide block: weight streaming, latency
        {"name": "ffn_decode_t1_d4096_f14336_bf16", "op": "ffn", "pass": "forward", "T": 1,
         "d": 4096, "f": 14336, "dtype": "bf16", "act": "silu"},
        # a batch of 24 decoding sequences through two fused 1408-wide shared experts
        {"name": "ffn_decode_t24_d2048_f2816_fp16", "op": "ffn", "pass": "forward", "T": 24,
         "d": 2048, "f": 2816, "dtype": "fp16", "act": "silu"},
        # the shared expert over a 4096-token prompt
        {"name": "ffn_prefill_t4096_d7168_f2048_bf16", "op": "ffn", "pass": "forward", "T": 4096,
         "d": 7168, "f": 2048, "dtype": "bf16", "act": "silu"},
        # a small fine-tuning step over a ragged number of tokens, fp16, GELU gate
        {"name": "ffn_train_t333_d2048_f1408_fp16", "op": "ffn", "pass": "train", "T": 333,
         "d": 2048, "f": 1408, "dtype": "fp16", "act": "gelu"},
        # a training step of the 14336-wide block over one 4096-token sequence
        {"name": "ffn_train_t4096_d4096_f14336_bf16", "op": "ffn", "pass": "train", "T": 4096,
         "d": 4096, "f": 14336, "dtype": "bf16", "act": "silu"},
        # the norm before the layer for one decoded token: launch latency
        {"name": "norm_rms_decode_r1_c7168_bf16", "op": "norm", "pass": "forward", "kind": "rms",
         "rows": 1, "cols": 7168, "dtype": "bf16", "wdtype": "bf16"},
        # the norm before the layer over a prompt
        {"name": "norm_layer_r4096_c7168_bf16", "op": "norm", "pass": "forward", "kind": "layer",
         "rows": 4096, "cols": 7168, "dtype": "bf16", "wdtype": "bf16"},
        # a training step's norm, fp32 parameters beside bf16 activations
        {"name": "norm_layer_train_r8192_c2048_bf16", "op": "norm", "pass": "train",
         "kind": "layer", "rows": 8192, "cols": 2048, "dtype": "bf16", "wdtype": "fp32"},
        # an odd width and a ragged batch: no aligned vector access on odd rows
        {"name": "norm_rms_train_r1777_c1003_fp16", "op": "norm", "pass": "train", "kind": "rms",
         "rows": 1777, "cols": 1003, "dtype": "fp16", "wdtype": "fp16"},
        # the residual of a small batch: launch latency
        {"name": "dropout_r128_c2048_bf16", "op": "dropout", "pass": "forward", "rows": 128,
         "cols": 2048, "dtype": "bf16", "p": 0.1},
        # a training step's residual add over a large batch
        {"name": "dropout_train_r8192_c7168_bf16", "op": "dropout", "pass": "train", "rows": 8192,
         "cols": 7168, "dtype": "bf16", "p": 0.1},
        # odd sizes in fp32
        {"name": "dropout_train_r777_c1001_fp32", "op": "dropout", "pass": "train", "rows": 777,
         "cols": 1001, "dtype": "fp32", "p": 0.25},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "norm", "dropout"])
    if op == "ffn":
        train = rng.random() < 0.5
        d = 8 * _log_int(rng, 16, 896)
        f = 8 * _log_int(rng, 8, 1792)
        per_token = (18 if train else 6) * d * f
        T = _log_int(rng, 1, max(1, min(8192, LARGEST_FLOPS // per_token)))
        return {"op": "ffn", "pass": "train" if train else "forward", "T": T, "d": d, "f": f,
                "dtype": rng.choice(["bf16", "fp16"]), "act": rng.choice(["silu", "gelu"])}
    cols = _log_int(rng, 64, 16384)
    rows = _log_int(rng, 1, max(1, min(16384, LARGEST_ELEMS // cols)))
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op == "norm":
        return {"op": "norm", "pass": rng.choice(["forward", "train"]),
                "kind": rng.choice(["layer", "rms"]), "rows": rows, "cols": cols, "dtype": dtype,
                "wdtype": rng.choice([dtype, "fp32"])}
    return {"op": "dropout", "pass": rng.choice(["forward", "train"]), "rows": rows,
            "cols": cols, "dtype": dtype, "p": rng.choice([0.0, 0.1, 0.25, 0.5])}


# ------------------------------------------------------------------------ inputs
def _inputs(case, seed):
    """The case's tensors on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        v = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return (v * scale + shift).to(dtype)

    train = case["pass"] == "train"
    if case["op"] == "ffn":
        T, d, f = case["T"], case["d"], case["f"]
        t = {"x": normal(T, d), "W1": normal(f, d, scale=d ** -0.5),
             "W3": normal(f, d, scale=d ** -0.5), "W2": normal(d, f, scale=f ** -0.5)}
        if train:
            t["dout"] = normal(T, d, scale=0.25)
        return t
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "norm":
        # a residual stream: rows of different scale, off their mean
        scale = 0.5 + 2 * torch.rand((rows, 1), generator=g, device="cuda")
        v = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
        t = {"x": ((v + 0.25) * scale).to(dt)}
        wdt = DTYPES[case["wdtype"]]
        t["weight"] = normal(cols, scale=0.1, shift=1.0, dtype=wdt)
        t["bias"] = normal(cols, scale=0.1, dtype=wdt) if case["kind"] == "layer" else None
        if train:
            t["dy"] = normal(rows, cols, scale=0.25)
        return t
    t = {"x": normal(rows, cols), "residual": normal(rows, cols, scale=2.0),
         # the generator's seed and offset, as a program keeps them on the device
         "rng": torch.randint(0, 2 ** 62, (2,), generator=g, device="cuda", dtype=torch.int64)}
    if train:
        t["dout"] = normal(rows, cols, scale=0.25)
    return t


EPS = 1e-5


def prepare(case, seed):
    return {"case": dict(case), **_inputs(case, seed)}


# ------------------------------------------------------------------------ plain forms
def _act_plain(a, name):
    """The gate's activation and its derivative, fp32."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-a))
        return a * s, s * (1 + a * (1 - s))
    c, k = math.sqrt(2 / math.pi), 0.044715          # GELU in its tanh form
    t = torch.tanh(c * (a + k * a ** 3))
    return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * c * (1 + 3 * k * a * a)


def _ffn_plain(s):
    dt, act = s["x"].dtype, s["case"]["act"]
    x, W1, W3, W2 = (s[k].float() for k in ("x", "W1", "W3", "W2"))
    gate, up = x @ W1.T, x @ W3.T
    a, da = _act_plain(gate, act)
    h = a * up
    out = h @ W2.T
    if s["case"]["pass"] == "forward":
        return out.to(dt)
    dout = s["dout"].float()
    dh = dout @ W2
    dgate, dup = dh * up * da, dh * a
    dx = dgate @ W1 + dup @ W3
    return {"out": out.to(dt), "dx": dx.to(dt), "dW1": (dgate.T @ x).to(dt),
            "dW3": (dup.T @ x).to(dt), "dW2": (dout.T @ h).to(dt)}


def _norm_plain(s):
    kind, x, w, b = s["case"]["kind"], s["x"].float(), s["weight"].float(), s["bias"]
    xc = x - x.mean(1, keepdim=True) if kind == "layer" else x
    rstd = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    xh = xc * rstd
    y = xh * w if b is None else xh * w + b.float()
    y = y.to(s["x"].dtype)
    if s["case"]["pass"] == "forward":
        return y
    dy = s["dy"].float()
    dxh = dy * w
    dx = dxh - xh * (dxh * xh).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - dxh.mean(1, keepdim=True)
    res = {"y": y, "dx": (dx * rstd).to(s["x"].dtype),
           "dweight": (dy * xh).double().sum(0).to(s["weight"].dtype)}
    if b is not None:
        res["dbias"] = dy.double().sum(0).to(b.dtype)
    return res


def _philox_plain(block, key, offset):
    """Philox-4x32-10 of the counters (block, offset): four 32-bit words each, int64."""
    m = 0xFFFFFFFF
    c0, c1 = block & m, (block >> 32) & m
    c2, c3 = (offset & m).expand_as(c0), ((offset >> 32) & m).expand_as(c0)
    k0, k1 = key & m, (key >> 32) & m
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((p1 >> 32) & m) ^ c1 ^ k0, p1 & m,
                          ((p0 >> 32) & m) ^ c3 ^ k1, p0 & m)
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return torch.stack((c0, c1, c2, c3), 1)


def _dropout_plain(s):
    x, p = s["x"], s["case"]["p"]
    n = x.numel()
    block = torch.arange((n + 3) // 4, device=x.device, dtype=torch.int64)
    words = _philox_plain(block, s["rng"][0], s["rng"][1]).reshape(-1)[:n].reshape(x.shape)
    keep = words >= round(p * 2 ** 32)
    scale = 1 / (1 - p)
    zero = torch.zeros((), device=x.device)
    out = (s["residual"].float() + torch.where(keep, x.float() * scale, zero)).to(x.dtype)
    if s["case"]["pass"] == "forward":
        return out
    dx = torch.where(keep, s["dout"].float() * scale, zero).to(x.dtype)
    return {"out": out, "dx": dx}


# ------------------------------------------------------------------------ one pass
def _run_own(s):
    from mixture_experts_ffn_expert_b200 import ops
    case = s["case"]
    train = case["pass"] == "train"
    if case["op"] == "ffn":
        if not train:
            return ops.gated_ffn_forward(s["x"], s["W1"], s["W3"], s["W2"],
                                         activation=case["act"])
        out, gate, up = ops.gated_ffn_forward(s["x"], s["W1"], s["W3"], s["W2"],
                                              activation=case["act"], save=True)
        dx, dW1, dW3, dW2 = ops.gated_ffn_backward(s["dout"], s["x"], s["W1"], s["W3"], s["W2"],
                                                   gate, up, activation=case["act"])
        return {"out": out, "dx": dx, "dW1": dW1, "dW3": dW3, "dW2": dW2}
    if case["op"] == "norm":
        if not train:
            return ops.norm_forward(s["x"], s["weight"], s["bias"], eps=EPS, kind=case["kind"])
        y, mean, rstd = ops.norm_forward(s["x"], s["weight"], s["bias"], eps=EPS,
                                         kind=case["kind"], save=True)
        dx, dweight, dbias = ops.norm_backward(s["dy"], s["x"], s["weight"], mean, rstd,
                                               kind=case["kind"], bias=s["bias"] is not None)
        res = {"y": y, "dx": dx, "dweight": dweight}
        if dbias is not None:
            res["dbias"] = dbias
        return res
    out = ops.dropout_add_forward(s["x"], s["residual"], case["p"], s["rng"])
    if not train:
        return out
    return {"out": out, "dx": ops.dropout_add_backward(s["dout"], case["p"], s["rng"])}


def run(state):
    if own:
        return _run_own(state)
    return {"ffn": _ffn_plain, "norm": _norm_plain, "dropout": _dropout_plain}[
        state["case"]["op"]](state)


# ------------------------------------------------------------------------ work
def work(case):
    """Bytes read and written once and operations of one pass."""
    b, train = BYTES[case["dtype"]], case["pass"] == "train"
    if case["op"] == "ffn":
        T, d, f = case["T"], case["d"], case["f"]
        if not train:
            return {"bytes": b * (2 * T * d + 3 * d * f), "flops": 6 * T * d * f}
        # x, dout, W in; out, dx, dW out
        return {"bytes": b * (4 * T * d + 6 * d * f), "flops": 18 * T * d * f}
    n = case["rows"] * case["cols"]
    if case["op"] == "norm":
        wb = BYTES[case["wdtype"]] * case["cols"] * (2 if case["kind"] == "layer" else 1)
        if not train:
            return {"bytes": 2 * n * b + wb, "flops": 8 * n}
        return {"bytes": 4 * n * b + 2 * wb, "flops": 24 * n}
    # Philox: 10 rounds of 2 wide products and 4 exclusive ors for 4 elements
    if not train:
        return {"bytes": 3 * n * b, "flops": 17 * n}
    return {"bytes": 5 * n * b, "flops": 33 * n}


# ------------------------------------------------------------------------ definition in 64 bits
def _mul_hi_lo(a, const):
    """High and low 32-bit halves of a 32-bit times a 32-bit number, in 16-bit limbs."""
    ah, al, ch, cl = a >> 16, a & 0xFFFF, const >> 16, const & 0xFFFF
    low = al * cl
    mid = ah * cl + (low >> 16)
    mid2 = al * ch + (mid & 0xFFFF)
    return ah * ch + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | (low & 0xFFFF)


def _keep_exact(n, p, seed, offset):
    ctr = [np.arange((n + 3) // 4, dtype=np.uint64), np.uint64(0), np.uint64(offset & 0xFFFFFFFF),
           np.uint64(offset >> 32)]
    ctr = [torch.as_tensor(np.broadcast_to(c, ctr[0].shape).astype(np.int64), device="cuda")
           for c in ctr]
    ctr[1], ctr[0] = torch.div(ctr[0], 2 ** 32, rounding_mode="floor"), ctr[0] % 2 ** 32
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for r in range(10):
        h0, l0 = _mul_hi_lo(ctr[0], 0xD2511F53)
        h1, l1 = _mul_hi_lo(ctr[2], 0xCD9E8D57)
        k0 = (key[0] + r * 0x9E3779B9) % 2 ** 32
        k1 = (key[1] + r * 0xBB67AE85) % 2 ** 32
        ctr = [h1 ^ ctr[1] ^ k0, l1, h0 ^ ctr[3] ^ k1, l0]
    words = torch.empty((ctr[0].numel(), 4), dtype=torch.int64, device="cuda")
    for i in range(4):
        words[:, i] = ctr[i]
    return ~(words.flatten()[:n] < int(round(p * 4294967296.0)))


def exact(case, seed):
    t = _inputs(case, seed)
    train = case["pass"] == "train"
    D = {k: v.double() for k, v in t.items() if v is not None and v.is_floating_point()}
    if case["op"] == "ffn":
        pre = D["x"].mm(D["W1"].t())
        up = D["x"].mm(D["W3"].t())
        if case["act"] == "silu":
            sg = torch.sigmoid(pre)
            val, der = pre * sg, sg + pre * sg * (1 - sg)
        else:
            # d/da [a/2 (1 + tanh(q(a)))], q = sqrt(2/pi) (a + 0.044715 a^3)
            q = math.sqrt(2 / math.pi) * (pre + 0.044715 * pre.pow(3))
            dq = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * pre.square())
            half = torch.sigmoid(2 * q)             # (1 + tanh q) / 2
            val, der = pre * half, half + pre * 2 * half * (1 - half) * dq
        out = (val * up).mm(D["W2"].t())
        if not train:
            return out
        back = D["dout"].mm(D["W2"])
        grads = {"out": out, "dW2": D["dout"].t().mm(val * up)}
        gate_grad, up_grad = back * up * der, back * val
        grads["dx"] = gate_grad.mm(D["W1"]) + up_grad.mm(D["W3"])
        grads["dW1"], grads["dW3"] = gate_grad.t().mm(D["x"]), up_grad.t().mm(D["x"])
        return {k: grads[k] for k in ("out", "dx", "dW1", "dW3", "dW2")}
    if case["op"] == "norm":
        x, w = D["x"], D["weight"]
        c = x.shape[1]
        mu = x.sum(1, keepdim=True) / c if case["kind"] == "layer" else torch.zeros_like(x[:, :1])
        inv = torch.rsqrt((x - mu).square().sum(1, keepdim=True) / c + EPS)
        xn = (x - mu) * inv
        y = xn * w + (D["bias"] if "bias" in D else 0.0)
        if not train:
            return y
        gy = D["dy"] * w
        dot = (gy * xn).sum(1, keepdim=True) / c
        dx = inv * (gy - xn * dot - (gy.sum(1, keepdim=True) / c if case["kind"] == "layer" else 0))
        res = {"y": y, "dx": dx, "dweight": torch.einsum("rc,rc->c", D["dy"], xn)}
        if "bias" in D:
            res["dbias"] = D["dy"].sum(0)
        return res
    seed_w, offset = (int(v) for v in t["rng"].tolist())
    keep = _keep_exact(t["x"].numel(), case["p"], seed_w, offset).view_as(t["x"])
    inv_keep = 1.0 / (1.0 - case["p"])
    out = D["residual"].clone()
    out[keep] += D["x"][keep] * inv_keep
    if not train:
        return out
    dx = torch.zeros_like(D["dout"])
    dx[keep] = D["dout"][keep] * inv_keep
    return {"out": out, "dx": dx}
