"""Operators of a transformer's feed-forward sublayer on gathered bf16 weights, in their plain form and through the library.

linear          y = residual + dropout(act(x W' + bias) * gate), optionally keeping z = x W' + bias
linear_dinput   da = dy W'^T, then the activation's (and gate's) gradient: dx = da * gate * act'(z), dgate = da * act(z)
linear_dweight  dw (+)= gradient of the weight, dbias (+)= sum of dy over the rows
dropout         y = residual + keep(x) / (1 - p), the mask from Philox4x32-10 at (column / 4, row, offset); its gradient is the same map on dy
norm            layer norm or RMS norm of each row, with the statistics its gradient needs
norm_backward   the input's gradient (plus the one that arrives over the residual branch) and the parameters' gradients

W' is w for weights kept as [k, n] (GPT-2) and its transpose for weights kept as [n, k] (Llama).
"""
import functools
import math

import numpy as np
import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
KINDS = ("linear", "linear_dinput", "linear_dweight", "dropout", "norm", "norm_backward")


def _linear(m, n, k, kn, act="none", bias="none", pre=False, gate=False, residual=False, p=0.0, out="bf16", pad=0):
    return {"op": "linear", "m": m, "n": n, "k": k, "kn": kn, "act": act, "bias": bias, "pre": pre, "gate": gate, "residual": residual, "p": p, "out": out, "pad": pad}


def _dinput(m, n, k, kn, act="none", gate=False, out="bf16", pad=0):
    return {"op": "linear_dinput", "m": m, "n": n, "k": k, "kn": kn, "act": act, "gate": gate, "out": out, "pad": pad}


def _dweight(m, n, k, kn, dbias=False, accumulate=False, out="bf16", pad=0):
    return {"op": "linear_dweight", "m": m, "n": n, "k": k, "kn": kn, "dbias": dbias, "accumulate": accumulate, "out": out, "pad": pad}


def _dropout(m, n, p, dtype="bf16", residual=False, pad=0):
    return {"op": "dropout", "m": m, "n": n, "p": p, "dtype": dtype, "residual": residual, "pad": pad}


def _norm(op, m, n, rms, dtype="bf16", params="bf16", dres=False, accumulate=False, pad=0):
    return {"op": op, "m": m, "n": n, "rms": rms, "dtype": dtype, "params": params, "dres": dres, "accumulate": accumulate, "pad": pad}


def listed():
    return [
        # one new token through GPT-2-medium's first feed-forward product: only the weight's bytes and the latency count
        dict(_linear(1, 4096, 1024, True, "gelu_tanh", "bf16"), name="token up 1024-4096"),
        # GPT-2-medium's second feed-forward product in training: bias, dropout and residual in one epilogue, 2 sequences of 1024
        dict(_linear(2048, 1024, 4096, True, "none", "bf16", residual=True, p=0.1), name="down 4096-1024 dropout"),
        # Llama-7B's gated product in training: silu(x Wg) times the up projection, z kept for the gradient; the largest case
        dict(_linear(4096, 11008, 4096, False, "silu", pre=True, gate=True), name="gate 4096-11008 silu"),
        # GPT-2-small's tied output projection in f32: an odd number of columns, rows that no 16-byte store fits
        dict(_linear(509, 50257, 768, False, out="f32"), name="logits 768-50257 f32"),
        # GPT-2-medium: the gradient through the second product and the GELU before it, 8 sequences
        dict(_dinput(8192, 1024, 4096, True, "gelu_tanh"), name="dinput 1024-4096 gelu"),
        # Llama-1.4B: the gradient through the down projection into both gated branches, a ragged batch of tokens
        dict(_dinput(1999, 2048, 5504, False, "silu", gate=True), name="dinput 2048-5504 gated"),
        # GPT-2-medium's first product: weight and bias gradients in bf16, added to those of the micro-batch before
        dict(_dweight(8192, 4096, 1024, True, dbias=True, accumulate=True), name="dweight 1024-4096 bias"),
        # Llama-1.4B's attention output: weight gradient in f32 for a ragged batch, a long sum into a small matrix
        dict(_dweight(6001, 2048, 2048, False, out="f32"), name="dweight 2048-2048 f32"),
        # GPT-2-medium's residual dropout over 16 sequences
        dict(_dropout(16384, 1024, 0.1, residual=True), name="dropout 16384x1024"),
        # a short f32 gradient with odd sizes
        dict(_dropout(257, 771, 0.25, dtype="f32"), name="dropout 257x771 f32"),
        # Llama-7B's RMS norm over a batch of 4 sequences of 2048
        dict(_norm("norm", 8192, 4096, True), name="rms norm 8192x4096"),
        # GPT-2-medium's layer norm backward: input and parameter gradients, the residual branch's gradient added
        dict(_norm("norm_backward", 8192, 1024, False, dres=True), name="layer norm grad 8192x1024"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    kind = rng.choice(("linear", "linear", "linear_dinput", "linear_dweight", "dropout", "norm", "norm_backward"))
    pad = rng.choice((0, 0, 8, 1))  # extra elements between rows
    out = rng.choice(("bf16", "bf16", "f32"))
    if kind.startswith("linear"):
        width = lambda: _log(rng, 64, 11008) if rng.random() < 0.5 else 8 * _log(rng, 8, 1376)  # noqa: E731
        m, n, k = _log(rng, 1, 8192), width(), width()
        while 2.0 * m * n * k > 2.4e11:
            m, n, k = _log(rng, 1, 8192), width(), width()
        kn, act = rng.random() < 0.5, rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
        if kind == "linear":
            return _linear(m, n, k, kn, act, rng.choice(("none", "bf16", "f32")), rng.random() < 0.4, rng.random() < 0.3, rng.random() < 0.4,
                           rng.choice((0.0, 0.0, 0.1, 0.5)), out, pad)
        if kind == "linear_dinput":
            return _dinput(m, n, k, kn, act, act != "none" and rng.random() < 0.4, "bf16" if act != "none" else out, pad)
        return _dweight(m, n, k, kn, rng.random() < 0.5, rng.random() < 0.4, out, pad)
    m, n = _log(rng, 1, 16384), _log(rng, 1, 12288)
    while m * n > (1 << 25):
        m, n = _log(rng, 1, 16384), _log(rng, 1, 12288)
    dtype = rng.choice(("bf16", "f32"))
    if kind == "dropout":
        return _dropout(m, n, rng.choice((0.1, 0.25, 0.5, 0.9)), dtype, rng.random() < 0.5, pad)
    n = max(n, 32)  # the gradient of a norm over a few elements cancels to nothing
    return _norm(kind, m, n, rng.random() < 0.5, dtype, rng.choice(("bf16", "f32")), kind == "norm_backward" and rng.random() < 0.5,
                 kind == "norm_backward" and rng.random() < 0.3, pad)


def _dtype(name):
    return F32 if name == "f32" else BF16


def _rows(c, m, n, dtype, g=None, scale=1.0, shift=0.0):
    """An [m, n] matrix whose rows lie n + pad elements apart; random where a generator is given."""
    if g is None:
        full = torch.zeros(m, n + c["pad"], dtype=dtype, device="cuda")
    else:
        full = torch.randn(m, n + c["pad"], dtype=F32, device="cuda", generator=g).mul_(scale).add_(shift).to(dtype)
    return full[:, :n]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    m, n, op = c["m"], c["n"], c["op"]
    vec = lambda size, dtype, scale, shift=0.0: torch.randn(size, device="cuda", generator=g).mul_(scale).add_(shift).to(dtype)  # noqa: E731
    if op.startswith("linear"):
        k = c["k"]
        w = lambda: _rows(c, *((k, n) if c["kn"] else (n, k)), BF16, g, 0.02)  # noqa: E731
    if op == "linear":
        c.update(x=_rows(c, m, k, BF16, g), w=w(), y=_rows(c, m, n, _dtype(c["out"])))
        c["b"] = None if c["bias"] == "none" else vec(n, _dtype(c["bias"]), 0.1)
        c["z"] = _rows(c, m, n, BF16) if c["pre"] else None
        c["u"] = _rows(c, m, n, BF16, g) if c["gate"] else None
        c["r"] = _rows(c, m, n, _dtype(c["out"]), g) if c["residual"] else None
    elif op == "linear_dinput":
        c.update(dy=_rows(c, m, n, BF16, g, 0.01), w=w(), dx=_rows(c, m, k, _dtype(c["out"])))
        c["z"] = _rows(c, m, k, BF16, g, 0.7) if c["act"] != "none" else None
        c["u"] = _rows(c, m, k, BF16, g) if c["gate"] else None
        c["du"] = _rows(c, m, k, BF16) if c["gate"] else None
    elif op == "linear_dweight":
        shape = (k, n) if c["kn"] else (n, k)
        c.update(dy=_rows(c, m, n, BF16, g, 0.01), x=_rows(c, m, k, BF16, g))
        c["dw"] = _rows(c, *shape, _dtype(c["out"]), g if c["accumulate"] else None, 0.1)
        c["db"] = (vec(n, _dtype(c["out"]), 0.1) if c["accumulate"] else torch.zeros(n, dtype=_dtype(c["out"]), device="cuda")) if c["dbias"] else None
    elif op == "dropout":
        d = _dtype(c["dtype"])
        c.update(x=_rows(c, m, n, d, g), y=_rows(c, m, n, d), r=_rows(c, m, n, d, g) if c["residual"] else None)
    else:
        d, q = _dtype(c["dtype"]), _dtype(c["params"])
        c.update(x=_rows(c, m, n, d, g, 1.0, 0.3), w=vec(n, q, 0.1, 1.0), b=None if c["rms"] else vec(n, q, 0.1))
        if op == "norm":
            c.update(y=_rows(c, m, n, d), mean=torch.empty(m, device="cuda"), rstd=torch.empty(m, device="cuda"))
        else:
            c.update(dy=_rows(c, m, n, d, g, 0.01), dx=_rows(c, m, n, d), r=_rows(c, m, n, d, g, 0.01) if c["dres"] else None)
            start = 0.1 if c["accumulate"] else 0.0
            c.update(dw=vec(n, q, start), db=None if c["rms"] else vec(n, q, start))
            x = c["x"].double()  # the statistics that the forward pass left
            mean = torch.zeros(m, dtype=torch.float64, device="cuda") if c["rms"] else x.mean(1)
            c.update(mean=mean.float(), rstd=((x - mean[:, None]).square().mean(1) + 1e-5).rsqrt().float())
            c["work"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")  # scratch that the program lends to its calls
    c["seed"], c["offset"] = 0x9E3779B97F4A7C15 ^ int(seed), (int(seed) * 977) & 0xFFFFFFFFFF
    return c


# ------------------------------------------------------------------ plain form
def _round(state, _):
    """One round of Philox4x32 on 32-bit words held in 64-bit integers."""
    a, b, c, d, k0, k1 = state
    p, q = a * 0xD2511F53, c * 0xCD9E8D57
    low = 0xFFFFFFFF
    return ((q >> 32) & low) ^ b ^ k0, q & low, ((p >> 32) & low) ^ d ^ k1, p & low, (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low


def _words(m, n, seed, offset, device):
    """The 32-bit word of each element of an [m, n] matrix."""
    low = 0xFFFFFFFF
    group = torch.arange((n + 3) // 4, device=device)[None, :].expand(m, -1)
    row = torch.arange(m, device=device)[:, None].expand(-1, group.shape[1])
    start = (group, row, torch.full_like(row, offset & low), torch.full_like(row, (offset >> 32) & low), seed & low, (seed >> 32) & low)
    a, b, c, d, _, _ = functools.reduce(_round, range(10), start)
    return torch.stack((a, b, c, d), -1).reshape(m, -1)[:, :n]


def _drop(v, p, seed, offset):
    p = np.float32(p)
    keep = _words(v.shape[0], v.shape[1], seed, offset, v.device) >= int(float(p) * 4294967296.0)
    return torch.where(keep, v * float(np.float32(1.0) / (np.float32(1.0) - p)), torch.zeros_like(v))


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _plain_linear(s):
    z = s["x"].float() @ (s["w"].float() if s["kn"] else s["w"].float().t())
    if s["b"] is not None:
        z = z + s["b"].float()
    v = _act(z, s["act"])
    if s["u"] is not None:
        v = v * s["u"].float()
    if s["p"]:
        v = _drop(v, s["p"], s["seed"], s["offset"])
    if s["r"] is not None:
        v = v + s["r"].float()
    return {"y": v.to(_dtype(s["out"])), "z": z.to(BF16) if s["pre"] else None}


def _plain_dinput(s):
    da = s["dy"].float() @ (s["w"].float().t() if s["kn"] else s["w"].float())
    if s["act"] == "none":
        return {"dx": da.to(_dtype(s["out"])), "dgate": None}
    z = s["z"].float()
    dx = da * _act_grad(z, s["act"])
    if s["u"] is None:
        return {"dx": dx.to(BF16), "dgate": None}
    return {"dx": (dx * s["u"].float()).to(BF16), "dgate": (da * _act(z, s["act"])).to(BF16)}


def _plain_dweight(s):
    dy, x = s["dy"].float(), s["x"].float()
    dw, db = x.t() @ dy if s["kn"] else dy.t() @ x, dy.sum(0) if s["dbias"] else None
    if s["accumulate"]:
        dw = dw + s["dw"].float()
        db = None if db is None else db + s["db"].float()
    s["dw"].copy_(dw)
    if db is not None:
        s["db"].copy_(db)
    return {"dw": s["dw"], "db": s["db"]}


def _plain_dropout(s):
    v = _drop(s["x"].float(), s["p"], s["seed"], s["offset"])
    return {"y": (v if s["r"] is None else v + s["r"].float()).to(_dtype(s["dtype"]))}


def _plain_norm(s):
    x = s["x"].float()
    mean = torch.zeros_like(x[:, 0]) if s["rms"] else x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(1) + 1e-5)
    y = c * rstd[:, None] * s["w"].float()
    y = y if s["rms"] else y + s["b"].float()
    return {"y": y.to(_dtype(s["dtype"])), "rstd": rstd, "mean": None if s["rms"] else mean}


def _plain_norm_backward(s):
    dy = s["dy"].float()
    h = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["w"].float()
    inner = g - h * (g * h).mean(1, keepdim=True)
    inner = inner if s["rms"] else inner - g.mean(1, keepdim=True)
    dx = inner * s["rstd"][:, None]
    dx = dx if s["r"] is None else dx + s["r"].float()
    dw, db = (dy * h).sum(0), None if s["rms"] else dy.sum(0)
    if s["accumulate"]:
        dw, db = dw + s["dw"].float(), None if db is None else db + s["db"].float()
    s["dw"].copy_(dw)
    if db is not None:
        s["db"].copy_(db)
    return {"dx": dx.to(_dtype(s["dtype"])), "dw": s["dw"], "db": s["db"]}


# ---------------------------------------------------------------- library form
def _library(s):
    import zero_sharded_optimizer_device_gb300 as Z

    m, n, op = s["m"], s["n"], s["op"]
    ld = lambda t: 0 if t is None else t.stride(0)  # noqa: E731
    kind = lambda name: Z.ZERO_F32 if name == "f32" else Z.ZERO_BF16  # noqa: E731
    acts = {"none": Z.ZERO_ACT_NONE, "relu": Z.ZERO_ACT_RELU, "gelu": Z.ZERO_ACT_GELU, "gelu_tanh": Z.ZERO_ACT_GELU_TANH, "silu": Z.ZERO_ACT_SILU}
    if op.startswith("linear"):
        k, layout, out = s["k"], Z.ZERO_W_KN if s["kn"] else Z.ZERO_W_NK, kind(s["out"])
    if op == "linear":
        drop = Z.dropout_rng(s["p"], s["seed"], s["offset"]) if s["p"] else None
        ep = Z.linear_epilogue(bias=s["b"], bias_dtype=kind(s["bias"]), act=acts[s["act"]], pre=s["z"], ldpre=ld(s["z"]), gate=s["u"], ldgate=ld(s["u"]),
                               residual=s["r"], ldres=ld(s["r"]), res_dtype=out, dropout=drop)
        Z.zero_linear(s["x"], ld(s["x"]), s["w"], ld(s["w"]), layout, m, n, k, ep, s["y"], ld(s["y"]), out)
        return {"y": s["y"], "z": s["z"]}
    if op == "linear_dinput":
        ag = None if s["act"] == "none" else Z.linear_act_grad(acts[s["act"]], s["z"], ld(s["z"]), gate=s["u"], ldgate=ld(s["u"]), dgate=s["du"], lddgate=ld(s["du"]))
        Z.zero_linear_dinput(s["dy"], ld(s["dy"]), s["w"], ld(s["w"]), layout, m, n, k, ag, s["dx"], ld(s["dx"]), out)
        return {"dx": s["dx"], "dgate": s["du"]}
    if op == "linear_dweight":
        Z.zero_linear_dweight(s["dy"], ld(s["dy"]), s["x"], ld(s["x"]), m, n, k, layout, s["dw"], ld(s["dw"]), out, s["db"], out, s["accumulate"])
        return {"dw": s["dw"], "db": s["db"]}
    data = kind(s["dtype"])
    if op == "dropout":
        Z.zero_dropout(s["x"], ld(s["x"]), data, s["r"], ld(s["r"]), data, m, n, Z.dropout_rng(s["p"], s["seed"], s["offset"]), s["y"], ld(s["y"]), data)
        return {"y": s["y"]}
    form, params = Z.ZERO_NORM_RMS if s["rms"] else Z.ZERO_NORM_LAYER, kind(s["params"])
    mean = None if s["rms"] else s["mean"]
    if op == "norm":
        Z.zero_layer_norm(s["x"], ld(s["x"]), data, s["w"], s["b"], params, m, n, form, 1e-5, s["y"], ld(s["y"]), data, mean, s["rstd"])
        return {"y": s["y"], "rstd": s["rstd"], "mean": mean}
    Z.zero_layer_norm_backward(s["dy"], ld(s["dy"]), data, s["x"], ld(s["x"]), data, s["w"], params, mean, s["rstd"], m, n, form, s["r"], ld(s["r"]),
                               s["dx"], ld(s["dx"]), data, s["dw"], s["db"], params, s["accumulate"], s["work"], s["work"].numel())
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def run(state):
    if own:
        return _library(state)
    plain = {"linear": _plain_linear, "linear_dinput": _plain_dinput, "linear_dweight": _plain_dweight, "dropout": _plain_dropout, "norm": _plain_norm,
             "norm_backward": _plain_norm_backward}
    return plain[state["op"]](state)


# ------------------------------------------------------------ what it comes to
def work(case):
    c = case
    m, n, op = c["m"], c["n"], c["op"]
    if op.startswith("linear"):
        k = c["k"]
        o = 4 if c["out"] == "f32" else 2
        flops = 2.0 * m * n * k
        if op == "linear":
            b = {"none": 0, "bf16": 2, "f32": 4}[c["bias"]]
            size = 2 * (m * k + n * k) + b * n + m * n * (o + 2 * c["pre"] + 2 * c["gate"] + o * c["residual"])
        elif op == "linear_dinput":
            size = 2 * (m * n + n * k) + m * k * (o + 2 * (c["act"] != "none") + 4 * c["gate"])
        else:
            size = 2 * (m * n + m * k) + (n * k + n * c["dbias"]) * o * (1 + c["accumulate"])
            flops += m * n * c["dbias"]
        return {"bytes": size, "flops": flops}
    d = 4 if c["dtype"] == "f32" else 2
    if op == "dropout":
        return {"bytes": m * n * d * (2 + c["residual"]), "flops": 2.0 * m * n}
    q = (4 if c["params"] == "f32" else 2) * (1 if c["rms"] else 2)
    if op == "norm":
        return {"bytes": 2 * m * n * d + q * n + m * (4 if c["rms"] else 8), "flops": 8.0 * m * n}
    return {"bytes": m * n * d * (3 + c["dres"]) + q * n * (1 + c["accumulate"]) + n * (4 if c["params"] == "f32" else 2) + m * (4 if c["rms"] else 8), "flops": 14.0 * m * n}


# --------------------------------------------------- the definition in 64 bits
def _mask64(m, n, p, seed, offset):
    """Keep (1) or drop (0) of each element: Philox4x32-10 by unsigned 64-bit arithmetic on the host, some rows at a time."""
    u, low, half = np.uint64, np.uint64(0xFFFFFFFF), np.uint64(32)
    groups, least = (n + 3) // 4, np.uint64(int(np.float64(np.float32(p)) * 2.0 ** 32))
    kept, some = np.empty((m, n), bool), max(1, 32768 // groups)
    for first in range(0, m, some):
        rows = min(some, m - first)
        ctr = [np.broadcast_to(np.arange(groups, dtype=u), (rows, groups)), np.broadcast_to(np.arange(first, first + rows, dtype=u)[:, None], (rows, groups)),
               np.full((rows, groups), offset & 0xFFFFFFFF, u), np.full((rows, groups), offset >> 32, u)]
        keys = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
        for _ in range(10):
            t0, t1 = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
            ctr = [(t1 >> half) ^ ctr[1] ^ u(keys[0]), t1 & low, (t0 >> half) ^ ctr[3] ^ u(keys[1]), t0 & low]
            keys = [(keys[0] + 0x9E3779B9) % 2 ** 32, (keys[1] + 0xBB67AE85) % 2 ** 32]
        kept[first:first + rows] = np.stack(ctr, axis=2).reshape(rows, 4 * groups)[:, :n] >= least
    return torch.from_numpy(kept).to("cuda").double()


def exact(case, seed):
    s = prepare(case, seed)
    m, n, op = s["m"], s["n"], s["op"]
    if op.startswith("linear") and 2.0 * m * n * s["k"] > 4e12:
        return None
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    rate = 1.0 / (1.0 - float(np.float32(s["p"]))) if "p" in s else 1.0
    drop = lambda v: v * _mask64(m, n, s["p"], s["seed"], s["offset"]) * rate if s["p"] else v  # noqa: E731

    def value_and_slope(z):
        if s["act"] == "relu":
            return torch.relu(z), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
        if s["act"] == "gelu":  # z times the normal distribution's mass below z
            mass = torch.special.ndtr(z)
            return z * mass, mass + z * torch.exp(z * z / -2) / math.sqrt(2 * math.pi)
        if s["act"] == "gelu_tanh":  # z times the logistic function of twice the cubic
            a, b = math.sqrt(8 / math.pi), 0.044715
            mass = torch.sigmoid(a * z + a * b * z ** 3)
            return z * mass, mass + z * mass * (1 - mass) * (a + 3 * a * b * z ** 2)
        if s["act"] == "silu":
            mass = torch.sigmoid(z)
            return z * mass, mass + z * mass * (1 - mass)
        return z, torch.ones_like(z)

    if op == "linear":
        z = torch.einsum("mk,kn->mn" if s["kn"] else "mk,nk->mn", s["x"], s["w"])
        z = z if s["b"] is None else z + s["b"]
        v = value_and_slope(z)[0] * (1.0 if s["u"] is None else s["u"])
        return {"y": drop(v) + (0.0 if s["r"] is None else s["r"]), "z": z if s["pre"] else None}
    if op == "linear_dinput":
        da = torch.einsum("mn,kn->mk" if s["kn"] else "mn,nk->mk", s["dy"], s["w"])
        if s["act"] == "none":
            return {"dx": da, "dgate": None}
        value, slope = value_and_slope(s["z"])
        return {"dx": da * slope * (1.0 if s["u"] is None else s["u"]), "dgate": None if s["u"] is None else da * value}
    if op == "linear_dweight":
        dw = torch.einsum("mk,mn->kn" if s["kn"] else "mk,mn->nk", s["x"], s["dy"])
        more = 1.0 if s["accumulate"] else 0.0
        return {"dw": dw + more * s["dw"], "db": torch.einsum("mn->n", s["dy"]) + more * s["db"] if s["dbias"] else None}
    if op == "dropout":
        return {"y": drop(s["x"]) + (0.0 if s["r"] is None else s["r"])}
    if op == "norm":
        mean = s["x"].sum(1) * (0.0 if s["rms"] else 1.0 / n)
        rstd = ((s["x"] - mean[:, None]).pow(2).sum(1) / n + 1e-5).pow(-0.5)
        y = torch.einsum("mn,m,n->mn", s["x"] - mean[:, None], rstd, s["w"]) + (0.0 if s["rms"] else s["b"])
        return {"y": y, "rstd": rstd, "mean": None if s["rms"] else mean}
    h = torch.einsum("mn,m->mn", s["x"] - s["mean"][:, None], s["rstd"])
    g = s["dy"] * s["w"]
    proj = torch.einsum("mn,mn->m", g, h) / n
    dx = torch.einsum("mn,m->mn", g - h * proj[:, None] - (0.0 if s["rms"] else g.mean(1, keepdim=True)), s["rstd"])
    more = 1.0 if s["accumulate"] else 0.0
    return {"dx": dx + (0.0 if s["r"] is None else s["r"]), "dw": torch.einsum("mn,mn->n", s["dy"], h) + more * s["dw"],
            "db": None if s["rms"] else s["dy"].sum(0) + more * s["db"]}
