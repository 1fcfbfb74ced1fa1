"""Updates by orthogonalised momentum and layers in microscaled 4-bit numbers, in their plain form and through the library.

orthogonalize   y = p_s(..p_1(x / (|x| + eps))), p(X) = a X + (b X X^T + c (X X^T)^2) X: Newton-Schulz steps towards the nearest matrix with orthonormal rows (columns)
muon_step       momentum <- mu momentum + g;  master <- (1 - lr wd) master - lr scale orthogonalize(g + mu momentum), on whole tensors of the flat buffers
fp4             x in E2M1 with one scale per block, along its rows and along its columns, and back: what 4-bit products read
fp4_linear      y = residual + act(x w^T + bias) * gate, x quantised in the call and w before; kept z = x w^T + bias
fp4_dinput      dx = dy w through the activation and gate that made the input, dy quantised in the call along the outputs
fp4_dweight     dw (+)= dy^T x, both quantised in the call along the rows

E2M1 holds 0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives. "mx": blocks of 32, scale 2^(floor(log2 amax) - 2).  "nv": blocks of 16, scale E4M3 of amax / (6 g),
g = amax of the whole / 2688.  Ties go to the even code, values past 6 to 6; nearest is taken of x / scale (mx), of fl(x fl(1 / fl(scale g))) in fp32 (nv).
"""
import math

import torch

own = False

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
JORDAN = (3.4445, -4.7750, 2.0315)


def _ortho(batch, m, n, dtype="bf16", steps=5, pad=0):
    return {"op": "orthogonalize", "batch": batch, "m": m, "n": n, "dtype": dtype, "steps": steps, "pad": pad}


def _muon(count, m, n, nesterov=True, decay=0.1, between=0, lr=4e-4, out="bf16"):
    return {"op": "muon_step", "batch": count, "m": m, "n": n, "nesterov": nesterov, "decay": decay, "between": between, "lr": lr, "steps": 5, "out": out}


def _fp4(m, n, form, dtype="bf16", both=True, out="bf16", pad=0):
    return {"op": "fp4", "m": m, "n": n, "form": form, "dtype": dtype, "both": both, "out": out, "pad": pad}


def _linear(m, n, k, form, act="none", bias=False, pre=False, gate=False, residual=False, out="bf16", pad=0):
    return {"op": "fp4_linear", "m": m, "n": n, "k": k, "form": form, "act": act, "bias": bias, "pre": pre, "gate": gate, "residual": residual, "out": out, "pad": pad}


def _dinput(m, n, k, form, act="none", gate=False, out="bf16", pad=0):
    return {"op": "fp4_dinput", "m": m, "n": n, "k": k, "form": form, "act": act, "gate": gate, "out": out, "pad": pad}


def _dweight(m, n, k, form, accumulate=False, out="bf16", pad=0):
    return {"op": "fp4_dweight", "m": m, "n": n, "k": k, "form": form, "accumulate": accumulate, "out": out, "pad": pad}


def listed():
    return [
        # one square projection of GPT-2-small: a chain of dependent small products, latency counts
        dict(_ortho(1, 768, 768), name="ortho 768x768"),
        # the square projections of all 24 layers of GPT-2-medium in one call, momentum in f32
        dict(_ortho(24, 1024, 1024, "f32"), name="ortho 24x1024x1024"),
        # Llama-7B's up projection, more rows than columns: the largest case
        dict(_ortho(1, 11008, 4096, "f32"), name="ortho 11008x4096"),
        # GPT-2-small's 12 attention projections, updated where they lie between their biases in the flat buffers
        dict(_muon(12, 768, 768, between=768), name="muon 12x768x768"),
        # Llama-1.4B: the down projections of four layers
        dict(_muon(4, 2048, 5504), name="muon 4x2048x5504"),
        # odd sizes at odd places of the flat buffers: no 16-byte access fits
        dict(_muon(3, 509, 771, nesterov=False, decay=0.0, between=5), name="muon 3x509x771"),
        # a batch of Llama-7B's activations for the forward product and for the weight's gradient
        dict(_fp4(8192, 4096, "nv"), name="fp4 nv 8192x4096"),
        # a small f32 matrix of odd sizes: blocks that end early in both directions
        dict(_fp4(257, 771, "mx", "f32", out="f32"), name="fp4 mx 257x771"),
        # one new token through Llama-7B's up projection: the weight's 4-bit codes and the latency count
        dict(_linear(1, 11008, 4096, "mx"), name="token 4096-11008 mx"),
        # Llama-7B's gated product in training: silu(z) times the up projection, z kept
        dict(_linear(4096, 11008, 4096, "nv", "silu", pre=True, gate=True), name="gate 4096-11008 nv"),
        # GPT-2-medium: the gradient through the second product and the GELU before it, 8 sequences of 1024
        dict(_dinput(8192, 1024, 4096, "mx", "gelu_tanh"), name="dinput 1024-4096 mx"),
        # Llama-1.4B's attention output: the weight's gradient of a ragged batch, added to that of the micro-batch before
        dict(_dweight(6001, 2048, 2048, "nv", accumulate=True, out="f32"), name="dweight 2048-2048 nv"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def _iteration_flops(c):
    k, far = min(c["m"], c["n"]), max(c["m"], c["n"])
    return c["batch"] * c["steps"] * (3.0 * k * k * far + 1.0 * k * k * k)  # the symmetric products need one triangle each


def draw(rng):
    kind = rng.choice(("orthogonalize", "muon_step", "fp4", "fp4_linear", "fp4_linear", "fp4_dinput", "fp4_dweight"))
    pad, out, form = rng.choice((0, 0, 8, 1)), rng.choice(("bf16", "bf16", "f32")), rng.choice(("mx", "nv"))
    if kind in ("orthogonalize", "muon_step"):
        side = lambda: _log(rng, 16, 8192) if rng.random() < 0.5 else 64 * _log(rng, 1, 128)  # noqa: E731
        c = None
        while c is None or _iteration_flops(c) > 1.5e12 or c["batch"] * c["m"] * c["n"] > (1 << 26):
            c = _ortho(_log(rng, 1, 32), side(), side(), rng.choice(("bf16", "f32")), rng.choice((5, 5, 5, 3, 6)), pad)
        if kind == "orthogonalize":
            return c
        return _muon(c["batch"], c["m"], c["n"], rng.random() < 0.7, rng.choice((0.0, 0.1, 0.01)), rng.choice((0, 16, 5, c["n"])), rng.choice((1e-4, 2e-4, 4e-4)), out)
    if kind == "fp4":
        m, n = _log(rng, 1, 16384), _log(rng, 1, 16384)
        while m * n > (1 << 25):
            m, n = _log(rng, 1, 16384), _log(rng, 1, 16384)
        return _fp4(m, n, form, rng.choice(("bf16", "f32")), rng.random() < 0.5, out, pad)
    width = lambda: _log(rng, 64, 11008) if rng.random() < 0.5 else 32 * _log(rng, 2, 344)  # noqa: E731
    m, n, k = _log(rng, 1, 8192), width(), width()
    while 2.0 * m * n * k > 3.6e11:
        m, n, k = _log(rng, 1, 8192), width(), width()
    act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
    if kind == "fp4_linear":
        return _linear(m, n, k, form, act, rng.random() < 0.4, rng.random() < 0.4, rng.random() < 0.3, rng.random() < 0.4, out, pad)
    if kind == "fp4_dinput":
        return _dinput(m, n, k, form, act, act != "none" and rng.random() < 0.4, "bf16" if act != "none" else out, pad)
    return _dweight(max(m, 64), n, k, form, rng.random() < 0.5, out, pad)


def _dtype(name):
    return F32 if name == "f32" else BF16


def _rows(c, m, n, dtype, g=None, scale=1.0):
    """An [m, n] matrix whose rows lie n + pad elements apart; random where a generator is given."""
    if g is None:
        full = torch.zeros(m, n + c["pad"], dtype=dtype, device="cuda")
    else:
        full = torch.randn(m, n + c["pad"], dtype=F32, device="cuda", generator=g).mul_(scale).to(dtype)
    return full[:, :n]


def _activations(c, m, n, dtype, g, scale=1.0):
    """The same with channels of unlike sizes, as activations have them."""
    x = _rows(c, m, n, F32, g, scale)
    return _layout(c, x * torch.randn(n, device="cuda", generator=g).mul_(0.7).exp_(), dtype)


def _layout(c, x, dtype):
    y = _rows(c, x.shape[-2], x.shape[-1], dtype)
    y.copy_(x)
    return y


def _gradients(batch, m, n, g):
    """Matrices like a layer's momentum: some strong directions over noise."""
    r = min(m, n, 48)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    strength = torch.arange(1, r + 1, device="cuda").float().pow(-0.7)
    return 1e-3 * (torch.bmm(rn(batch, m, r) * strength, rn(batch, r, n)) + 0.5 * rn(batch, m, n))


def _places(c):
    """First elements of a muon_step's tensors in the flat buffers, and the buffers' length."""
    each = c["m"] * c["n"] + c["between"]
    total = c["batch"] * each + 1
    return [1 + t * each for t in range(c["batch"])] if c["between"] % 2 else [t * each for t in range(c["batch"])], (total + 127) // 128 * 128


def _packed_bytes(rows, cols, form):
    blocks = -(-cols // (16 if form == "nv" else 32))
    return -(-cols // 32) * 16, -(-rows // 128) * -(-blocks // 4) * 512


def _room(rows, cols, form):
    """Buffers that a program keeps for a quantised matrix."""
    row, scales = _packed_bytes(rows, cols, form)
    return {"codes": torch.zeros(rows, row, dtype=torch.uint8, device="cuda"), "scales": torch.zeros(scales, dtype=torch.uint8, device="cuda"),
            "g": torch.ones(1, device="cuda") if form == "nv" else None}


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    m, n, op = c["m"], c["n"], c["op"]
    if op == "orthogonalize":
        full = torch.zeros(c["batch"], m, n + c["pad"], dtype=_dtype(c["dtype"]), device="cuda")
        c["x"] = full[:, :, :n]
        c["x"].copy_(_gradients(c["batch"], m, n, g))
        c["y"] = torch.zeros(c["batch"], m, n + c["pad"], dtype=BF16, device="cuda")[:, :, :n]
    elif op == "muon_step":
        places, total = _places(c)
        new = lambda scale: torch.randn(total, device="cuda", generator=g).mul_(scale)  # noqa: E731
        c.update(master=new(0.02), momentum=new(0.0), reduced=new(1e-3), out=torch.zeros(total, dtype=_dtype(c["out"]), device="cuda"))
        size = m * n
        grads, old = _gradients(c["batch"], m, n, g), _gradients(c["batch"], m, n, g)
        for t, at in enumerate(places):
            c["reduced"][at:at + size] = 8 * grads[t].reshape(-1)  # a sum over 8 ranks
            c["momentum"][at:at + size] = 10 * old[t].reshape(-1)
        c["coef"] = torch.full((1,), 0.7, device="cuda")  # what the global norm left of the gradient
    elif op == "fp4":
        c["x"] = _activations(c, m, n, _dtype(c["dtype"]), g)
        c["q"], c["qt"] = _room(m, n, c["form"]), _room(n, m, c["form"]) if c["both"] else None
        c["y"], c["yt"] = _rows(c, m, n, _dtype(c["out"])), _rows(c, n, m, _dtype(c["out"])) if c["both"] else None
    elif op == "fp4_linear":
        k = c["k"]
        c.update(x=_activations(c, m, k, BF16, g), q=_room(m, k, c["form"]), y=_rows(c, m, n, _dtype(c["out"])))
        c["w"] = _pack(torch.randn(n, k, device="cuda", generator=g).mul_(0.02), c["form"])
        c["b"] = torch.randn(n, device="cuda", generator=g).mul_(0.1).to(BF16) if c["bias"] else None
        c["z"] = _rows(c, m, n, BF16) if c["pre"] else None
        c["u"] = _rows(c, m, n, BF16, g) if c["gate"] else None
        c["r"] = _rows(c, m, n, _dtype(c["out"]), g) if c["residual"] else None
    elif op == "fp4_dinput":
        k = c["k"]
        c.update(x=_activations(c, m, n, BF16, g, 0.01), q=_room(m, n, c["form"]), y=_rows(c, m, k, _dtype(c["out"])))
        c["w"] = _pack(torch.randn(k, n, device="cuda", generator=g).mul_(0.02), c["form"])
        c["z"] = _rows(c, m, k, BF16, g, 0.7) if c["act"] != "none" else None
        c["u"] = _rows(c, m, k, BF16, g) if c["gate"] else None
        c["du"] = _rows(c, m, k, BF16) if c["gate"] else None
    else:
        k = c["k"]
        c.update(dy=_activations(c, m, n, BF16, g, 0.01), x=_activations(c, m, k, BF16, g), q=_room(n, m, c["form"]), qx=_room(k, m, c["form"]))
        c["dw"] = _rows(c, n, k, _dtype(c["out"]), g if c["accumulate"] else None, 0.1)
    return c


# ------------------------------------------------------------------ plain form
def _iterate(x, steps):
    """Newton-Schulz steps on [batch, m, n]."""
    a, b, c = JORDAN
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + 1e-7)
    for _ in range(steps):
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.transpose(1, 2) if tall else x


def _plain_orthogonalize(s):
    s["y"].copy_(_iterate(s["x"].float(), s["steps"]))
    return {"y": s["y"]}


MU, SCALE = 0.95, 0.2  # momentum; the update's size, as a share of Adam's, times sqrt(the longer side)


def _plain_muon(s):
    m, n = s["m"], s["n"]
    at = torch.tensor(_places(s)[0], device="cuda")[:, None] + torch.arange(m * n, device="cuda")
    grad = s["reduced"][at] * 0.125 * s["coef"]
    mom = MU * s["momentum"][at] + grad
    u = grad + MU * mom if s["nesterov"] else mom
    step = _iterate(u.reshape(-1, m, n), s["steps"]).reshape(-1, m * n)
    w = s["master"][at]
    w = w - s["lr"] * s["decay"] * w - s["lr"] * SCALE * math.sqrt(max(m, n)) * step
    s["momentum"][at], s["master"][at], s["out"][at] = mom, w, w.to(s["out"].dtype)
    return {"momentum": s["momentum"], "master": s["master"], "out": s["out"]}


def _power(e):
    """2^e in 64 bits, by its exponent's bits: exp2 need not be exact."""
    return ((e.long() + 1023) << 52).view(F64)


def _tensor_scale(x):
    """g of a matrix in form nv."""
    a = x.abs()
    a = torch.where(torch.isfinite(a), a, torch.zeros_like(a)).max()
    return torch.where(a > 0, a / torch.full_like(a, 2688.0), torch.ones_like(a))  # (by a number, torch multiplies with its reciprocal)


def _blocks(x, size):
    return torch.nn.functional.pad(x, (0, -x.shape[1] % size)).reshape(x.shape[0], -1, size)


def _quantise(x, form, g):
    """Of an f32 matrix: signed E2M1 values by block and each block's scale (a byte and what it stands for)."""
    b = _blocks(x, 16 if form == "nv" else 32)
    amax = b.abs().amax(2)
    if form == "nv":
        s = (amax / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        byte, s = s.view(torch.uint8), s.float()
        d = s * g
        r = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    else:
        e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
        e = torch.where(amax > 0, e, torch.full_like(e, -127))
        byte, s, r = (e + 127).to(torch.uint8), _power(e).float(), _power(-e).float()
    q = b * r[:, :, None]
    a = q.abs()
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return code, q < 0, byte, s


LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(code, negative, s, cols):
    v = torch.tensor(LEVELS, device="cuda")[code]
    v = torch.where(negative, -v, v) * s[:, :, None]
    return v.reshape(v.shape[0], -1)[:, :cols]


def _pack(w, form):
    """A weight as a program keeps it: two codes a byte (the even column in the low half), rows of whole 16 bytes; scales in tiles of 128 rows and 4 blocks, row r of
    a tile at byte 16 (r % 32) + 4 (r / 32)."""
    g = _tensor_scale(w).reshape(1) if form == "nv" else None
    code, negative, byte, _ = _quantise(w, form, g)
    rows = w.shape[0]
    nibble = _blocks((code + 8 * negative.int()).reshape(rows, -1)[:, :w.shape[1]], 32).reshape(rows, -1).to(torch.uint8)
    codes = nibble[:, 0::2] + 16 * nibble[:, 1::2]
    tiles = torch.nn.functional.pad(byte, (0, -byte.shape[1] % 4, 0, -rows % 128))
    tiles = tiles.reshape(tiles.shape[0] // 128, 4, 32, tiles.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return {"codes": codes.contiguous(), "scales": tiles.contiguous().reshape(-1), "g": g}


def _unpack(p, rows, cols, form):
    """What the packed codes and scales stand for, without g."""
    nibble = torch.stack((p["codes"] & 15, p["codes"] >> 4), 2).reshape(rows, -1).int()
    size = 16 if form == "nv" else 32
    blocks = -(-cols // size)
    byte = p["scales"].reshape(-(-rows // 128), -1, 32, 4, 4).permute(0, 3, 2, 1, 4)
    byte = byte.reshape(byte.shape[0] * 128, -1)[:rows, :blocks].contiguous()
    s = byte.view(torch.float8_e4m3fn).float() if form == "nv" else _power(byte.int() - 127).float()
    nibble = _blocks(nibble[:, :cols], size)
    return _values(nibble & 7, nibble > 7, s, cols)


def _scaled(x, form):
    """x as its codes and scales stand for it, without g, and g."""
    g = _tensor_scale(x).reshape(1) if form == "nv" else None
    code, negative, _, s = _quantise(x, form, g)
    return _values(code, negative, s, x.shape[1]), g


def _back(x, form):
    """x through E2M1: with d = fl(scale g) a value is fl(code d)."""
    g = _tensor_scale(x).reshape(1) if form == "nv" else None
    code, negative, _, s = _quantise(x, form, g)
    return _values(code, negative, s * g if form == "nv" else s, x.shape[1])


def _plain_fp4(s):
    x = s["x"].float()
    s["y"].copy_(_back(x, s["form"]))
    if s["both"]:
        s["yt"].copy_(_back(x.t().contiguous(), s["form"]))
    return {"y": s["y"], "yt": s["yt"]}


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


def _product(x, w, gx, gw):
    z = x @ w.t()
    return z if gx is None else z * (gx * gw)


def _plain_linear(s):
    x, gx = _scaled(s["x"].float(), s["form"])
    z = _product(x, _unpack(s["w"], s["n"], s["k"], s["form"]), gx, s["w"]["g"])
    z = z if s["b"] is None else z + s["b"].float()
    v = _act(z, s["act"])
    v = v if s["u"] is None else v * s["u"].float()
    v = v if s["r"] is None else v + s["r"].float()
    s["y"].copy_(v)
    if s["pre"]:
        s["z"].copy_(z)
    return {"y": s["y"], "z": s["z"]}


def _plain_dinput(s):
    dy, gy = _scaled(s["x"].float(), s["form"])
    da = _product(dy, _unpack(s["w"], s["k"], s["n"], s["form"]), gy, s["w"]["g"])
    if s["act"] == "none":
        s["y"].copy_(da)
        return {"dx": s["y"], "dgate": None}
    z = s["z"].float()
    dx = da * _act_grad(z, s["act"])
    s["y"].copy_(dx if s["u"] is None else dx * s["u"].float())
    if s["u"] is not None:
        s["du"].copy_(da * _act(z, s["act"]))
    return {"dx": s["y"], "dgate": s["du"]}


def _plain_dweight(s):
    dy, gy = _scaled(s["dy"].float().t().contiguous(), s["form"])
    x, gx = _scaled(s["x"].float().t().contiguous(), s["form"])
    dw = _product(dy, x, gy, gx)
    s["dw"].copy_(dw + s["dw"].float() if s["accumulate"] else dw)
    return {"dw": s["dw"]}


# ---------------------------------------------------------------- library form
def _library(s):
    import zero_sharded_optimizer_device_gb300 as Z

    m, n, op = s["m"], s["n"], s["op"]
    ld = lambda t: 0 if t is None else t.stride(-2)  # noqa: E731
    kind = lambda t: Z.ZERO_F32 if t.dtype == F32 else Z.ZERO_BF16  # noqa: E731

    def scratch(size):  # lent by the program, kept between its calls
        if "work" not in s or s["work"].numel() < size:
            s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        return s["work"]

    if op == "orthogonalize":
        size = Z.zero_orthogonalize_workspace(m, n, s["batch"])
        Z.zero_orthogonalize(s["x"], ld(s["x"]), s["x"].stride(0), kind(s["x"]), m, n, s["batch"], Z.newton_schulz(s["steps"], JORDAN, 1e-7),
                             s["y"], ld(s["y"]), s["y"].stride(0), scratch(size), size)
        return {"y": s["y"]}
    if op == "muon_step":
        if "plan" not in s:  # made once by the program; one tensor of each layer is updated here, a bias lies between two
            odd = s["between"] % 2
            each = [m * n] + [s["between"]] * (s["between"] > 0)
            numels = [1] * odd + each * s["batch"]
            s["plan"] = Z.zero_plan(numels + [len(s["master"]) - sum(numels)] * (len(s["master"]) > sum(numels)), 8, 16)
            s["tensors"] = [odd + t * len(each) for t in range(s["batch"])]
        size = Z.zero_muon_workspace(m, n, s["batch"])
        hp = Z.muon_hp(lr=s["lr"], momentum=MU, weight_decay=s["decay"], grad_scale=0.125, nesterov=s["nesterov"], scale=SCALE * math.sqrt(max(m, n)),
                       ns=Z.newton_schulz(s["steps"], JORDAN, 1e-7))
        Z.zero_muon_step(s["plan"], s["tensors"], m, n, s["master"], s["momentum"], s["reduced"], hp, s["coef"], s["out"], kind(s["out"]), scratch(size), size)
        return {"momentum": s["momentum"], "master": s["master"], "out": s["out"]}

    form = Z.ZERO_FP4_NV if s["form"] == "nv" else Z.ZERO_FP4_MX
    packed = lambda q: None if q is None else Z.fp4_matrix(q["codes"], q["codes"].stride(0), q["scales"], q["g"])  # noqa: E731

    def quantise(x, q, qt, rows, cols):
        for other in (q, qt):
            if form == Z.ZERO_FP4_NV and other is not None:
                other["g"] = (q or qt)["g"]
        if form == Z.ZERO_FP4_NV:
            Z.zero_fp4_tensor_scale(x, ld(x), kind(x), rows, cols, (q or qt)["g"], scratch(Z.ZERO_FP4_WORKSPACE), Z.ZERO_FP4_WORKSPACE)
        q, qt = packed(q), packed(qt)
        Z.zero_fp4_quantize(x, ld(x), kind(x), rows, cols, form, q, qt)
        return q, qt

    acts = {"none": Z.ZERO_ACT_NONE, "relu": Z.ZERO_ACT_RELU, "gelu": Z.ZERO_ACT_GELU, "gelu_tanh": Z.ZERO_ACT_GELU_TANH, "silu": Z.ZERO_ACT_SILU}
    if op == "fp4":
        q, qt = quantise(s["x"], s["q"], s["qt"], m, n)
        Z.zero_fp4_dequantize(q, m, n, form, s["y"], ld(s["y"]), kind(s["y"]))
        if s["both"]:
            Z.zero_fp4_dequantize(qt, n, m, form, s["yt"], ld(s["yt"]), kind(s["yt"]))
        return {"y": s["y"], "yt": s["yt"]}
    k = s["k"]
    if op == "fp4_linear":
        q, _ = quantise(s["x"], s["q"], None, m, k)
        ep = Z.linear_epilogue(bias=s["b"], act=acts[s["act"]], pre=s["z"], ldpre=ld(s["z"]), gate=s["u"], ldgate=ld(s["u"]), residual=s["r"], ldres=ld(s["r"]),
                               res_dtype=kind(s["y"]))
        Z.zero_fp4_linear(q, packed(s["w"]), form, m, n, k, ep, s["y"], ld(s["y"]), kind(s["y"]))
        return {"y": s["y"], "z": s["z"]}
    if op == "fp4_dinput":
        q, _ = quantise(s["x"], s["q"], None, m, n)
        ag = None if s["act"] == "none" else Z.linear_act_grad(acts[s["act"]], s["z"], ld(s["z"]), gate=s["u"], ldgate=ld(s["u"]), dgate=s["du"], lddgate=ld(s["du"]))
        Z.zero_fp4_linear_dinput(q, packed(s["w"]), form, m, n, k, ag, s["y"], ld(s["y"]), kind(s["y"]))
        return {"dx": s["y"], "dgate": s["du"]}
    _, dy = quantise(s["dy"], None, s["q"], m, n)
    _, x = quantise(s["x"], None, s["qx"], m, k)
    Z.zero_fp4_linear_dweight(dy, x, form, m, n, k, s["dw"], ld(s["dw"]), kind(s["dw"]), s["accumulate"])
    return {"dw": s["dw"]}


def run(state):
    if own:
        return _library(state)
    plain = {"orthogonalize": _plain_orthogonalize, "muon_step": _plain_muon, "fp4": _plain_fp4, "fp4_linear": _plain_linear, "fp4_dinput": _plain_dinput,
             "fp4_dweight": _plain_dweight}
    return plain[state["op"]](state)


# ------------------------------------------------------------ what it comes to
def work(case):
    c = case
    m, n, op = c["m"], c["n"], c["op"]
    size = lambda name: 4 if name == "f32" else 2  # noqa: E731
    if op == "orthogonalize":
        return {"bytes": c["batch"] * m * n * (size(c["dtype"]) + 2), "flops": _iteration_flops(c)}
    if op == "muon_step":  # gradient read; momentum and master read and written; parameters written
        return {"bytes": c["batch"] * m * n * (20 + size(c["out"])), "flops": _iteration_flops(c)}
    packed = lambda r, q: _packed_bytes(r, q, c["form"])[1] + r * q / 2  # noqa: E731
    if op == "fp4":  # codes written, then read to go back
        ways = 2 if c["both"] else 1
        return {"bytes": m * n * (size(c["dtype"]) + ways * size(c["out"])) + 2 * (packed(m, n) + (packed(n, m) if c["both"] else 0)), "flops": 4.0 * m * n * ways}
    k, o = c["k"], size(c["out"])
    flops = 2.0 * m * n * k
    if op == "fp4_linear":  # the activations are read in bf16; their codes are the call's own
        return {"bytes": 2 * m * k + packed(n, k) + m * n * (o + 2 * c["pre"] + 2 * c["gate"] + o * c["residual"]) + 2 * n * c["bias"], "flops": flops}
    if op == "fp4_dinput":
        return {"bytes": 2 * m * n + packed(k, n) + m * k * (o + 2 * (c["act"] != "none") + 4 * c["gate"]), "flops": flops}
    return {"bytes": 2 * m * (n + k) + n * k * o * (1 + c["accumulate"]), "flops": flops}


# --------------------------------------------------- the definition in 64 bits
def _orthogonal64(x, steps):
    """The steps of each matrix, a X + b G X + c G^2 X with the Gram matrix G of the shorter side; the constants are the fp32 values that a call passes."""
    a, b, c = (float(torch.tensor(v, dtype=F32)) for v in JORDAN)
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + float(torch.tensor(1e-7, dtype=F32)))
    for _ in range(steps):
        if x.shape[1] <= x.shape[2]:
            gram = torch.einsum("bij,bkj->bik", x, x)
            x = a * x + b * torch.einsum("bik,bkj->bij", gram, x) + c * torch.einsum("bik,bkj->bij", torch.einsum("bik,bkl->bil", gram, gram), x)
        else:
            gram = torch.einsum("bji,bjk->bik", x, x)
            x = a * x + b * torch.einsum("bji,bik->bjk", x, gram) + c * torch.einsum("bji,bik->bjk", x, torch.einsum("bik,bkl->bil", gram, gram))
    return x


def _nearest64(x, form):
    """x [rows, cols] in 64 bits through E2M1 by rounding in steps of .5, 1 or 2; the roundings to fp32 are the definition's. Returns the values without g, and g."""
    size, rows, cols = (16 if form == "nv" else 32), x.shape[0], x.shape[1]
    f = lambda v: v.float().double()  # noqa: E731
    full = torch.zeros(rows, (cols + size - 1) // size * size, dtype=F64, device=x.device)
    full[:, :cols] = x
    full = full.unfold(1, size, size)
    top, g = full.abs().max(2).values, torch.ones((), dtype=F64, device=x.device)
    if form == "nv":
        g = f(x.abs().max() / 2688)
        t = f(top / f(6 * g)).clamp_max(448)
        grain = _power(torch.frexp(t.clamp_min(2.0 ** -6))[1] - 4)
        s = torch.round(t / grain) * grain
        one = f(s * g)
        scaled = f(full * torch.where(one > 0, f(1 / one.clamp_min(1e-300)), 0 * one)[:, :, None])
    else:
        s = _power(torch.frexp(top.clamp_min(2.0 ** -125))[1] - 3)
        scaled = full / s[:, :, None]
    a = scaled.abs()
    grain = 0.5 + 0.5 * (a >= 2) + 1.0 * (a >= 4)
    v = torch.sign(scaled) * (torch.round(a / grain) * grain).clamp_max(6)
    return (v * s[:, :, None]).flatten(1)[:, :cols], g


def exact(case, seed):
    s = prepare(case, seed)
    m, n, op = s["m"], s["n"], s["op"]
    if op == "orthogonalize":
        return {"y": _orthogonal64(s["x"].double(), s["steps"])}
    if op == "muon_step":
        momentum, master, out = s["momentum"].double(), s["master"].double(), s["out"].double()
        f = lambda v: float(torch.tensor(v, dtype=F32))  # noqa: E731
        spans = [slice(at, at + m * n) for at in _places(s)[0]]
        grads = [s["reduced"][p].double() / 8 * s["coef"].double() for p in spans]
        for p, grad in zip(spans, grads):
            momentum[p] = f(MU) * momentum[p] + grad
        u = torch.stack([grad + f(MU) * momentum[p] if s["nesterov"] else momentum[p] for p, grad in zip(spans, grads)]).reshape(-1, m, n)
        for p, step in zip(spans, _orthogonal64(u, s["steps"])):
            master[p] = master[p] * (1 - f(s["lr"]) * f(s["decay"])) - f(s["lr"]) * f(SCALE * math.sqrt(max(m, n))) * step.reshape(-1)
            out[p] = master[p]
        return {"momentum": momentum, "master": master, "out": out}
    form = s["form"]
    if op == "fp4":
        both = [_nearest64(v, form) for v in ((s["x"].double(), s["x"].double().t()) if s["both"] else (s["x"].double(),))]
        values = [v * g for v, g in both]
        return {"y": values[0], "yt": values[1] if s["both"] else None}
    if op == "fp4_dweight":
        (dy, gy), (x, gx) = _nearest64(s["dy"].double().t(), form), _nearest64(s["x"].double().t(), form)
        return {"dw": torch.einsum("nm,km->nk", dy * gy, x * gx) + (s["dw"].double() if s["accumulate"] else 0.0)}
    k = s["k"]
    g = torch.Generator(device="cuda").manual_seed(int(seed))  # the weight as it was before it was packed: drawn after the activations, as prepare does
    if op == "fp4_linear":
        _activations(s, m, k, BF16, g)
        w = torch.randn(n, k, device="cuda", generator=g).mul_(0.02)
    else:
        _activations(s, m, n, BF16, g, 0.01)
        w = torch.randn(k, n, device="cuda", generator=g).mul_(0.02)
    (x, gx), (w, gw) = _nearest64(s["x"].double(), form), _nearest64(w.double(), form)
    z = torch.einsum("ab,cb->ac", x, w) * (gx * gw)

    def value_and_slope(z):
        if s["act"] == "relu":
            return torch.relu(z), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
        if s["act"] == "gelu":  # z times the normal distribution's mass below z
            mass = torch.special.ndtr(z)
            return z * mass, mass + z * torch.exp(z * z / -2) / math.sqrt(2 * math.pi)
        if s["act"] == "gelu_tanh":  # z times the logistic function of twice the cubic
            p, q = math.sqrt(8 / math.pi), 0.044715
            mass = torch.sigmoid(p * z + p * q * z ** 3)
            return z * mass, mass + z * mass * (1 - mass) * (p + 3 * p * q * z ** 2)
        if s["act"] == "silu":
            mass = torch.sigmoid(z)
            return z * mass, mass + z * mass * (1 - mass)
        return z, torch.ones_like(z)

    if op == "fp4_linear":
        z = z if s["b"] is None else z + s["b"].double()
        v = value_and_slope(z)[0] * (1.0 if s["u"] is None else s["u"].double())
        return {"y": v + (0.0 if s["r"] is None else s["r"].double()), "z": z if s["pre"] else None}
    if s["act"] == "none":
        return {"dx": z, "dgate": None}
    value, slope = value_and_slope(s["z"].double())
    return {"dx": z * slope * (1.0 if s["u"] is None else s["u"].double()), "dgate": None if s["u"] is None else z * value}
