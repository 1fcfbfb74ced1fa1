"""The layer operators in 64 bits on the CPU, written from their formulas, and
bounds on how far an fp32 computation rounded once may lie from them.  Inputs
are torch tensors holding the very values the kernels read."""
import math

import numpy as np
import torch

D = torch.float64
U32 = 2.0 ** -23          # one fp32 rounding, to nearest or towards zero
U16 = 2.0 ** -8           # one bf16 rounding, to nearest: half of 2^-7 of its power of two
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def philox(ctr, key):
    """Philox4x32-10 on uint64 arrays holding 32-bit words: ctr 4, key 2."""
    u = np.uint64
    c, k = [np.asarray(v, u) for v in ctr], [int(v) for v in key]
    m32 = u(0xFFFFFFFF)
    for _ in range(10):
        p, q = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(q >> u(32)) ^ c[1] ^ u(k[0]), q & m32, (p >> u(32)) ^ c[3] ^ u(k[1]), p & m32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep_mask(m, n, p, seed, offset):
    """bool [m, n]: which elements dropout keeps."""
    g = (n + 3) // 4
    col = np.tile(np.arange(g, dtype=np.uint64), (m, 1))
    row = np.tile(np.arange(m, dtype=np.uint64)[:, None], (1, g))
    off = offset % 2 ** 64
    w = philox([col, row, np.full((m, g), off & 0xFFFFFFFF), np.full((m, g), off >> 32)],
               [seed & 0xFFFFFFFF, seed >> 32])
    words = np.stack(w, -1).reshape(m, 4 * g)[:, :n]
    return torch.from_numpy(words.astype(np.float64) >= math.floor(float(np.float32(p)) * 2.0 ** 32))


def drop(v, p, seed, offset):
    if p == 1.0:
        return torch.zeros_like(v)
    mask = keep_mask(v.shape[0], v.shape[1], p, seed, offset)
    return torch.where(mask, v / (1.0 - float(np.float32(p))), torch.zeros_like(v))


def act(z, name):
    """(act(z), act'(z))"""
    one = torch.ones_like(z)
    if name == "relu":
        return torch.where(z < 0, 0 * one, z), torch.where(z > 0, one, 0 * one)
    if name == "gelu":
        phi = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        cdf = torch.erfc(-z / math.sqrt(2)) / 2
        return z * cdf, cdf + z * phi
    if name == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        t, du = torch.tanh(u), math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
        return z * (1 + t) / 2, (1 + t) / 2 + z * (1 - t * t) * du / 2
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s + z * s * (1 - s)
    return z, one


def weight(w, kn):
    """The k x n matrix of a stored weight."""
    return w.to(D) if kn else w.to(D).T


def linear(x, w, kn, bias=None, a="none", gate=None, p=None, seed=0, offset=0, residual=None):
    """(y, z, error): error bounds |fp32 computation - y| before the final rounding."""
    x, w = x.to(D), weight(w, kn)
    z, size = x @ w, x.abs() @ w.abs()
    if bias is not None:
        z, size = z + bias.to(D), size + bias.to(D).abs()
    dz = (x.shape[1] + 4) * U32 * size
    v, _ = act(z, a)
    # every slope is below 1.13; the functions' own error is a few fp32 ulps of z
    dv = 1.13 * dz + (0 if a == "none" else 32 * U32 * z.abs())
    if gate is not None:
        v, dv = v * gate.to(D), dv * gate.to(D).abs() + 2 * U32 * (v * gate.to(D)).abs()
    if p is not None:
        v, dv = drop(v, p, seed, offset), dv / max(1e-30, 1 - p) + 4 * U32 * v.abs() / max(1e-30, 1 - p)
    if residual is not None:
        v = v + residual.to(D)
        dv = dv + 2 * U32 * v.abs()
    return v, z, dv, dz


def linear_dinput(dy, w, kn, a=None, pre=None, gate=None):
    """(dx, dgate, error of dx, error of dgate)"""
    dy, w = dy.to(D), weight(w, kn)
    da, err = dy @ w.T, (dy.shape[1] + 4) * U32 * (dy.abs() @ w.T.abs())
    if a is None:
        return da, None, err, None
    v, s = act(pre.to(D), a)
    g = 1.0 if gate is None else gate.to(D)
    size = s.abs() + 32 * U32 * (1 + pre.to(D).abs())
    dx = da * s * g
    ex = (err * size + da.abs() * 32 * U32 * (1 + pre.to(D).abs())) * (abs(g) if gate is not None else 1.0)
    if gate is None:
        return dx, None, ex, None
    return dx, da * v, ex, err * (v.abs() + 1e-6) + da.abs() * 32 * U32 * pre.to(D).abs()


def linear_dweight(dy, x, kn, dw0=None, db0=None):
    """(dw, db, error of dw, error of db)"""
    dy, x = dy.to(D), x.to(D)
    dw, e = (x.T @ dy, x.T.abs() @ dy.abs()) if kn else (dy.T @ x, dy.T.abs() @ x.abs())
    db, f = dy.sum(0), dy.abs().sum(0)
    if dw0 is not None:
        dw, e = dw + dw0.to(D), e + dw0.to(D).abs()
    if db0 is not None:
        db, f = db + db0.to(D), f + db0.to(D).abs()
    c = (dy.shape[0] + 4) * U32
    return dw, db, c * e, c * f


def norm(x, w, b, rms, eps):
    """(y, mean, rstd, error of y)"""
    x, w = x.to(D), w.to(D)
    n = x.shape[1]
    mean = torch.zeros(x.shape[0], dtype=D) if rms else x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / (c.square().mean(1) + eps).sqrt()
    y = c * rstd[:, None] * w
    # sums of n values in fp32: the mean is off by up to n ulps of the mean size (pairwise and
    # blocked sums stay far below), the distances by as much, rstd by half their relative error
    size = x.abs().mean(1)
    depth = 16 + math.log2(n + 1) + n / 256
    dmean = 0 * size if rms else depth * U32 * size
    dc = dmean[:, None] + U32 * c.abs()
    drel = depth * U32 + 2 * dmean * rstd + 4 * U32
    err = (dc * rstd[:, None] + c.abs() * rstd[:, None] * drel[:, None]) * w.abs()
    if b is not None:
        y = y + b.to(D)
        err = err + U32 * (y.abs() + b.to(D).abs())
    return y, mean, rstd, err


def norm_backward(dy, x, w, mean, rstd, rms, dres=None, dw0=None, db0=None):
    """(dx, dw, db, error of dx, error of dw, error of db)"""
    dy, x, w = dy.to(D), x.to(D), w.to(D)
    n, m = x.shape[1], x.shape[0]
    mean = torch.zeros(m, dtype=D) if mean is None else mean.to(D)
    r = rstd.to(D)[:, None]
    h = (x - mean[:, None]) * r
    g = dy * w
    mg = 0 * r if rms else g.mean(1, keepdim=True)
    mgh = (g * h).mean(1, keepdim=True)
    dx = r * (g - mg - h * mgh)
    depth = 24 + math.log2(n + 1) + n / 256
    size = g.abs() + g.abs().mean(1, keepdim=True) + h.abs() * (g * h).abs().mean(1, keepdim=True)
    dh = U32 * (x.abs() + mean.abs()[:, None]) * r + U32 * h.abs()      # x - mean cancels
    ex = r * (depth * U32 * size + dh * mgh.abs() + h.abs() * (g.abs() * dh).mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.to(D)
        ex = ex + 2 * U32 * dx.abs()
    dw, db = (dy * h).sum(0), dy.sum(0)
    rows = (m + 16) * U32
    ew = rows * (dy * h).abs().sum(0) + (dy.abs() * dh).sum(0)
    eb = rows * dy.abs().sum(0)
    if dw0 is not None:
        dw, ew = dw + dw0.to(D), ew + 2 * U32 * dw0.to(D).abs()
    if db0 is not None:
        db, eb = db + db0.to(D), eb + 2 * U32 * db0.to(D).abs()
    return dx, dw, db, ex, ew, eb


def assert_within(got, want, err, what):
    """|got - want| <= the computation's error and one rounding to got's dtype."""
    u = U16 if got.dtype == torch.bfloat16 else U32
    got, tol = got.detach().cpu().to(D), err + u * (want.abs() + err) + 1e-37
    off = (got - want).abs()
    bad = ~(off <= tol)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements outside their "
                             f"bound, first at {i}: got {got[i]:.9g} want {want[i]:.9g} "
                             f"bound {tol[i]:.3g}")
