"""The training operators that stand between the FP4 linears, as measured work:
layer normalisation with its backward pass, dropout without a stored mask, the
two fused with the residual addition, and the backward pass of the SwiGLU
activation.

With ``own`` false, ``run`` computes each operator from elementary torch
operations in binary32 (sums over the rows in binary64), rounded once at the
end; with ``own`` true it makes the calls a training program makes.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5
DROP_TAG = 0x44524F50  # word 3 of the dropout counters
MOST_BYTES = 5 * 2 * 8192 * 14336  # the largest listed case


# ---------------------------------------------------------------- cases ---
def _norm(name, op, rows, cols, dtype="bf16", weight="same", bias=True, center=True, pad=0):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "weight": weight,
            "bias": bias, "center": center, "pad": pad}


def listed():
    return [
        # one token of a 4096-wide model: latency alone
        _norm("norm 1x4096", "norm_fwd", 1, 4096),
        # the norm before the 8B block's linears, one training step's tokens
        _norm("norm 8192x4096", "norm_fwd", 8192, 4096),
        # RMS form on odd binary32 rows: nothing is aligned
        _norm("rms norm fp32 777x4099", "norm_fwd", 777, 4099, "fp32", bias=False, center=False),
        # its backward pass, the residual stream's gradient joining it
        dict(_norm("norm bwd 8192x4096", "norm_bwd", 8192, 4096), dres=True),
        # a norm as wide as the MLP, fp16 activations with binary32 weights
        dict(_norm("norm bwd fp16 1000x14336", "norm_bwd", 1000, 14336, "fp16", weight="fp32"),
             dres=False),
        # dropout of a small batch, without residual
        {"name": "dropout 33x4096", "op": "drop_fwd", "rows": 33, "cols": 4096, "dtype": "bf16",
         "p": 0.1, "residual": False, "pad": 0},
        # dropout of a sub-layer's output into the residual stream (the stack's 16384 tokens)
        {"name": "dropout+res 16384x4096", "op": "drop_fwd", "rows": 16384, "cols": 4096,
         "dtype": "bf16", "p": 0.1, "residual": True, "pad": 0},
        # its backward pass on odd binary32 rows with a padded leading dimension
        {"name": "dropout bwd fp32 2047x6145", "op": "drop_bwd", "rows": 2047, "cols": 6145,
         "dtype": "fp32", "p": 0.5, "residual": False, "pad": 3},
        # dropout, residual and norm in one pass: what a block does twice per step
        dict(_norm("drop+res+norm 8192x4096", "fused_fwd", 8192, 4096), p=0.1),
        dict(_norm("drop+res+norm bwd 8192x4096", "fused_bwd", 8192, 4096), p=0.1),
        # the gated MLP's activation, backward: a ragged small batch and a training step
        {"name": "swiglu bwd 96x14336", "op": "swiglu_bwd", "rows": 96, "cols": 14336},
        {"name": "swiglu bwd 8192x14336", "op": "swiglu_bwd", "rows": 8192, "cols": 14336},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "drop_fwd", "drop_bwd", "fused_fwd", "fused_bwd",
                     "swiglu_bwd"])
    rows, cols = _log(rng, 1, 16384), _log(rng, 64, 28672)
    if op == "swiglu_bwd":
        cols = max(32, min(cols, 14336) // 32 * 32)
        return {"op": op, "rows": max(1, min(rows, MOST_BYTES // (10 * cols))), "cols": cols}
    if rng.random() < 0.7:
        cols = max(8, cols // 8 * 8)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    rows = max(1, min(rows, MOST_BYTES // (5 * SIZE[dtype] * cols)))
    pad = rng.choice([0, 0, 8, rng.randint(1, 40)])
    case = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "pad": pad}
    if op.startswith("drop"):
        return dict(case, p=rng.choice([0.05, 0.1, 0.25, 0.5]),
                    residual=op == "drop_fwd" and rng.random() < 0.5)
    case.update(weight=rng.choice(["same", "fp32"]), bias=rng.random() < 0.6,
                center=rng.random() < 0.6)
    if op == "norm_bwd":
        case["dres"] = rng.random() < 0.5
    if op.startswith("fused"):
        case["p"] = rng.choice([0.05, 0.1, 0.25, 0.5])
    return case


# --------------------------------------------------------------- inputs ---
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows, cols = case["rows"], case["cols"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def matrix(x, dtype, pad):
        """x in `dtype` as a program holds it: rows `pad` elements apart."""
        held = torch.zeros(rows, x.shape[1] + pad, dtype=dtype, device="cuda")
        held[:, :x.shape[1]] = x
        return held[:, :x.shape[1]]

    if case["op"] == "swiglu_bwd":
        gate, up, grad = randn(rows, cols), randn(rows, cols), randn(rows, cols)
        return {"case": case, "z": torch.cat([gate * 1.5, up], 1).bfloat16(),
                "dh": (grad * 1e-3 * randn(rows, 1).exp()).bfloat16()}
    dtype, pad = DTYPES[case["dtype"]], case["pad"]
    st = {"case": case, "seed": 0x9E3779B97F4A7C15 ^ seed,
          "step": torch.full((1,), 1000 + seed % 1000, dtype=torch.int64, device="cuda")}

    def activation():
        """N(0, 1) with a mean of its own per channel and outlier channels."""
        x = randn(rows, cols) + 0.1 * randn(1, cols)
        return x * torch.where(torch.rand(1, cols, generator=g, device="cuda") < 0.005, 20.0, 1.0)

    def gradient():
        return randn(rows, cols) * 1e-3 * randn(rows, 1).exp()

    def weights():
        wd = torch.float32 if case["weight"] == "fp32" else dtype
        st["w"] = (1.0 + 0.2 * randn(cols)).to(wd)
        st["b"] = (0.1 * randn(cols)).to(wd) if case["bias"] else None

    if case["op"] in ("norm_fwd", "drop_fwd", "fused_fwd"):
        st["x"] = matrix(activation(), dtype, pad)
        if case["op"] == "fused_fwd" or case.get("residual"):
            st["res"] = matrix(activation(), dtype, pad)
        if case["op"] != "drop_fwd":
            weights()
    elif case["op"] == "drop_bwd":
        st["dy"] = matrix(gradient(), dtype, pad)
    else:
        st["x"] = matrix(activation(), dtype, pad)
        st["dy"] = matrix(gradient(), dtype, pad)
        if case["op"] == "fused_bwd" or case["dres"]:
            st["ds"] = matrix(gradient(), dtype, pad)
        weights()
        x = st["x"].double()
        mean = x.mean(1) if case["center"] else torch.zeros(rows, device="cuda", dtype=torch.float64)
        st["rstd"] = ((x - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        st["mean"] = mean.float() if case["center"] else None
    return st


# ----------------------------------------------------------- plain forms ---
def _philox_plain(key, rows, groups):
    """Philox4x32-7 (Salmon et al., SC'11) on counters (group, row, 0, tag):
    four words [rows, groups] of 32 bits each, in int64."""
    m = 0xFFFFFFFF
    dev = key.device
    c = [torch.arange(groups, device=dev).expand(rows, groups),
         torch.arange(rows, device=dev)[:, None].expand(rows, groups),
         torch.zeros((), dtype=torch.int64, device=dev),
         torch.full((), DROP_TAG, dtype=torch.int64, device=dev)]
    k0, k1 = key & m, (key >> 32) & m
    # seven rounds; the int64 product wraps, its 64 bits are the right ones
    for _ in range(7):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((p1 >> 32) & m) ^ c[1] ^ k0, p1 & m, ((p0 >> 32) & m) ^ c[3] ^ k1, p0 & m]
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return c


def _threshold(p):
    return min(round(p * 65536), 65535)


def _signed64(v):
    v &= (1 << 64) - 1
    return v - (1 << 64) if v >> 63 else v


def _kept_plain(st, rows, cols):
    key = st["step"][0] + _signed64(st["seed"])
    words = torch.stack(_philox_plain(key, rows, (cols + 7) // 8), -1)
    u = torch.stack([words & 0xFFFF, words >> 16], -1).reshape(rows, -1)[:, :cols]
    return u >= _threshold(st["case"]["p"])


def _drop_plain(st, x):
    t = _threshold(st["case"]["p"])
    return torch.where(_kept_plain(st, *x.shape), x * (65536 / (65536 - t)), 0.0)


def _norm_plain(st, x):
    case = st["case"]
    x = x.float()
    mean = x.mean(1) if case["center"] else None
    xc = x - mean[:, None] if case["center"] else x
    rstd = 1.0 / torch.sqrt(xc.square().mean(1) + EPS)
    y = xc * rstd[:, None] * st["w"].float()
    if st["b"] is not None:
        y = y + st["b"].float()
    return y, mean, rstd


def _norm_bwd_plain(st):
    case, dy, x, rstd = st["case"], st["dy"].float(), st["x"].float(), st["rstd"][:, None]
    xh = (x - st["mean"][:, None]) * rstd if case["center"] else x * rstd
    wdy = dy * st["w"].float()
    inner = wdy - xh * (wdy * xh).mean(1, keepdim=True)
    if case["center"]:
        inner = inner - wdy.mean(1, keepdim=True)
    dx = inner * rstd
    if "ds" in st:
        dx = dx + st["ds"].float()
    dw = (dy * xh).sum(0, dtype=torch.float64).float()
    db = dy.sum(0, dtype=torch.float64).float() if case["bias"] else None
    return dx, dw, db


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "swiglu_bwd":
        f = case["cols"]
        gate, up, dh = st["z"][:, :f].float(), st["z"][:, f:].float(), st["dh"].float()
        sig = 1.0 / (1.0 + torch.exp(-gate))
        dgate = dh * up * sig * (1.0 + gate * (1.0 - sig))
        return [torch.cat([dgate, dh * gate * sig], 1).bfloat16()]
    dtype = DTYPES[case["dtype"]]
    if op == "norm_fwd":
        y, mean, rstd = _norm_plain(st, st["x"])
        return [y.to(dtype), mean, rstd]
    if op == "norm_bwd":
        dx, dw, db = _norm_bwd_plain(st)
        return [dx.to(dtype), dw, db]
    if op == "drop_fwd":
        y = _drop_plain(st, st["x"].float())
        return [(st["res"].float() + y if "res" in st else y).to(dtype)]
    if op == "drop_bwd":
        return [_drop_plain(st, st["dy"].float()).to(dtype)]
    if op == "fused_fwd":
        s = (st["res"].float() + _drop_plain(st, st["x"].float())).to(dtype)
        y, mean, rstd = _norm_plain(st, s)  # the norm is that of the stored s
        return [y.to(dtype), s, mean, rstd]
    ds, dw, db = _norm_bwd_plain(st)
    return [_drop_plain(st, ds).to(dtype), ds.to(dtype), dw, db]


# ---------------------------------------------------- the framework's calls ---
def _own(st):
    import fp4_quantization_block_b200 as fa
    case = st["case"]
    op = case["op"]
    if op == "swiglu_bwd":
        return [fa.swiglu_bwd(st["z"], st["dh"])]
    if op == "norm_fwd":
        return list(fa.layer_norm_fwd(st["x"], st["w"], st["b"], eps=EPS, center=case["center"]))
    if op == "norm_bwd":
        return list(fa.layer_norm_bwd(st["dy"], st["x"], st["w"], st["mean"], st["rstd"],
                                      center=case["center"], bias_grad=case["bias"],
                                      dres=st.get("ds")))
    if op == "drop_fwd":
        return [fa.dropout_fwd(st["x"], case["p"], st["seed"], step=st["step"],
                               residual=st.get("res"))]
    if op == "drop_bwd":
        return [fa.dropout_bwd(st["dy"], case["p"], st["seed"], step=st["step"])]
    if op == "fused_fwd":
        return list(fa.dropout_add_layer_norm_fwd(
            st["x"], st["res"], st["w"], st["b"], case["p"], st["seed"], step=st["step"], eps=EPS,
            center=case["center"]))
    return list(fa.dropout_add_layer_norm_bwd(
        st["dy"], st["ds"], st["x"], st["w"], st["mean"], st["rstd"], case["p"], st["seed"],
        step=st["step"], center=case["center"], bias_grad=case["bias"]))


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------- work ---
def work(case):
    e = case["rows"] * case["cols"]
    op = case["op"]
    if op == "swiglu_bwd":
        return {"bytes": 10 * e, "flops": 14 * e}
    b = SIZE[case["dtype"]]
    if op.startswith("drop"):
        return {"bytes": (3 if case["residual"] else 2) * b * e, "flops": 2 * e}
    wb = 4 if case["weight"] == "fp32" else b
    nb = 2 if case["bias"] else 1
    stats = 4 * case["rows"] * (2 if case["center"] else 1)
    if op.endswith("fwd"):
        arrays, small = (2 if op == "norm_fwd" else 4), nb * wb * case["cols"]
        return {"bytes": arrays * b * e + small + stats, "flops": 8 * e}
    arrays = 5 if op == "fused_bwd" else 4 if case["dres"] else 3
    return {"bytes": arrays * b * e + (wb + 4 * nb) * case["cols"] + stats, "flops": 14 * e}


# ---------------------------------------------------------------- exact ---
def _kept_exact(seed, step, p, rows, cols):
    """The kept elements by Philox4x32-7 in numpy, on unsigned words."""
    u32, u64 = np.uint32, np.uint64
    key = (seed + step) & ((1 << 64) - 1)
    ka, kb = key & 0xFFFFFFFF, key >> 32
    groups = -(-cols // 8)
    a = np.tile(np.arange(groups, dtype=u32), rows)
    b = np.repeat(np.arange(rows, dtype=u32), groups)
    c, d = np.zeros_like(a), np.full_like(a, DROP_TAG)
    for i in range(7):
        x, y = a.astype(u64) * u64(0xD2511F53), c.astype(u64) * u64(0xCD9E8D57)
        ra, rb = (ka + i * 0x9E3779B9) & 0xFFFFFFFF, (kb + i * 0xBB67AE85) & 0xFFFFFFFF
        a, c = (y >> u64(32)).astype(u32) ^ b ^ u32(ra), (x >> u64(32)).astype(u32) ^ d ^ u32(rb)
        b, d = y.astype(u32), x.astype(u32)
    bits = np.stack([a, b, c, d], -1).view(np.uint16)  # little endian: low half first
    t = min(int(np.rint(p * 65536.0)), 65535)
    kept = bits.reshape(rows, groups * 8)[:, :cols] >= t
    return torch.from_numpy(np.ascontiguousarray(kept)).cuda(), 65536 / (65536 - t)


def exact(case, seed):
    st = prepare(case, seed)
    op, n = case["op"], case["cols"]
    if op == "swiglu_bwd":
        gate, up = st["z"].double().chunk(2, 1)
        dh = st["dh"].double()
        sig = torch.sigmoid(gate)
        silu = gate * sig
        return [torch.hstack([dh * up * (sig + silu * torch.sigmoid(-gate)), dh * silu])]
    dtype = DTYPES[case["dtype"]]

    def drop(v):
        kept, scale = _kept_exact(st["seed"], int(st["step"]), case["p"], *v.shape)
        return (v * scale).masked_fill(~kept, 0.0)

    def norm(v):
        mu = v.sum(1, keepdim=True) / n if case["center"] else v.new_zeros(len(v), 1)
        r = ((v - mu).pow(2).sum(1, keepdim=True) / n + EPS).pow(-0.5)
        y = torch.addcmul(st["b"].double() if case["bias"] else v.new_zeros(n), (v - mu) * r,
                          st["w"].double())
        return y, (mu[:, 0] if case["center"] else None), r[:, 0]

    def norm_bwd():
        dy, r = st["dy"].double(), st["rstd"].double()[:, None]
        xh = st["x"].double()
        if case["center"]:
            xh = xh - st["mean"].double()[:, None]
        xh = xh * r
        dxh = dy * st["w"].double()
        along = torch.einsum("ij,ij->i", dxh, xh)[:, None]
        level = dxh.sum(1, keepdim=True) if case["center"] else 0.0
        dx = (n * dxh - level - xh * along) * (r / n)
        if "ds" in st:
            dx += st["ds"].double()
        return dx, torch.einsum("ij,ij->j", dy, xh), dy.sum(0) if case["bias"] else None

    if op == "norm_fwd":
        return list(norm(st["x"].double()))
    if op == "norm_bwd":
        return list(norm_bwd())
    if op == "drop_fwd":
        y = drop(st["x"].double())
        return [y + st["res"].double() if "res" in st else y]
    if op == "drop_bwd":
        return [drop(st["dy"].double())]
    if op == "fused_fwd":
        s = drop(st["x"].double()) + st["res"].double()
        y, mean, rstd = norm(s.to(dtype).double())
        return [y, s, mean, rstd]
    ds, dw, db = norm_bwd()
    return [drop(ds), ds, dw, db]
