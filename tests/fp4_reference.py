"""Microscaled 4-bit numbers on the CPU in 64 bits, written from their
definition; the roundings to fp32 that the definition names are made as such."""
import torch

D, F = torch.float64, torch.float32
LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=D)
SIZE = {"mx": 32, "nv": 16}


def f32(v):
    """A double rounded to fp32."""
    return v.to(F).to(D)


def e4m3(byte):
    """What E4M3 bytes (sign bit clear) stand for: 127 is NaN."""
    byte = byte.to(torch.int64)
    e, m = byte >> 3, (byte & 7).to(D)
    v = torch.where(e > 0, (1 + m / 8) * torch.pow(torch.tensor(2.0, dtype=D), (e - 7).to(D)), m / 8 * 2.0 ** -6)
    return torch.where(byte == 127, torch.full_like(v, float("nan")), v)


E4M3 = e4m3(torch.arange(127))


def nearest_byte(t):
    """The nearest E4M3's byte, ties to the even one, beyond 448 to 448."""
    t = t.clamp(max=448.0)
    hi = torch.searchsorted(E4M3, t.contiguous()).clamp(max=126)   # the first that is not below
    lo = (hi - 1).clamp(min=0)
    up, down = E4M3[hi] - t, t - E4M3[lo]
    return torch.where(up < down, hi, torch.where(down < up, lo, torch.where(lo % 2 == 0, lo, hi))).to(torch.uint8)


def nearest_code(q):
    """The nearest level's code of |q|, ties to the even code."""
    a = q.abs().clamp(max=8.0)                                     # (differences of huge values would all be the same)
    gap = (a[..., None] - LEVELS).abs()
    best = gap.amin(-1, keepdim=True)
    tied = gap == best                                             # one or two neighbours
    even = tied & (torch.arange(8) % 2 == 0)
    pick = torch.where(even.any(-1, keepdim=True), even, tied)
    return pick.to(torch.uint8).argmax(-1).to(torch.uint8)


def tensor_scale(x):
    a = x.to(D).abs()
    a = a[torch.isfinite(a)]
    top = a.max() if a.numel() else torch.tensor(0.0, dtype=D)
    return f32(top / 2688) if top > 0 else torch.tensor(1.0, dtype=D)


def quantise(x, form, g=None):
    """(codes [rows, cols], scale bytes [rows, blocks], values [rows, cols]) of x, in double exactly."""
    size, rows, cols = SIZE[form], x.shape[0], x.shape[1]
    g = torch.tensor(1.0, dtype=D) if g is None else g.to(D)
    full = torch.zeros(rows, -(-cols // size) * size, dtype=D)
    full[:, :cols] = x.to(D)
    b = full.reshape(rows, -1, size)
    bad = ~torch.isfinite(b).all(2)
    fine = torch.where(bad[..., None], torch.zeros_like(b), b)
    top = fine.abs().amax(2)
    if form == "nv":
        byte = nearest_byte(f32(top / f32(6 * g)))
        d = f32(E4M3[byte.long()] * g)
        r = torch.where(d > 0, f32(1 / torch.where(d > 0, d, torch.ones_like(d))), torch.zeros_like(d))
        q = f32(fine * r[..., None])
        value = d
    else:
        e = torch.where(top > 0, torch.frexp(torch.where(top > 0, top, torch.ones_like(top)))[1] - 3, torch.full(top.shape, -127, dtype=torch.int32)).clamp(min=-127)
        byte = (e + 127).to(torch.uint8)
        value = torch.ldexp(torch.ones_like(top), e)
        q = fine / value[..., None]
    code = nearest_code(q)
    v = f32(LEVELS[code.long()] * value[..., None])
    v = torch.where(torch.signbit(fine), -v, v)
    code = code + 8 * torch.signbit(fine).to(torch.uint8)
    byte = torch.where(bad, torch.full_like(byte, 127 if form == "nv" else 255), byte)
    code = torch.where(bad[..., None], torch.zeros_like(code), code)
    v = torch.where(bad[..., None], torch.full_like(v, float("nan")), v)
    flat = lambda t: t.reshape(rows, -1)[:, :cols].contiguous()  # noqa: E731
    return flat(code), byte, flat(v)


def size(rows, cols, form):
    blocks = -(-cols // SIZE[form])
    return -(-cols // 32) * 16, -(-rows // 128) * -(-blocks // 4) * 512


def pack(code, byte, form):
    """(codes [rows, row bytes], scales [bytes]) in memory's layout, written out element by element from its description."""
    rows, cols = code.shape
    row_bytes, scale_bytes = size(rows, cols, form)
    wide = torch.zeros(rows, 2 * row_bytes, dtype=torch.uint8)
    wide[:, :cols] = code
    out = torch.zeros(scale_bytes, dtype=torch.uint8)
    blocks = byte.shape[1]
    r, b = torch.meshgrid(torch.arange(rows), torch.arange(blocks), indexing="ij")
    at = ((r // 128) * -(-blocks // 4) + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4
    out[at.reshape(-1)] = byte.reshape(-1)
    return wide[:, 0::2] | wide[:, 1::2] << 4, out
