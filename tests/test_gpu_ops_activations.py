"""The activations and their slopes at every bf16 value, in relative terms.

A product with one input and a weight of 1 hands each bf16 value z to the
epilogue exactly, so what is off is the activation's.  The bounds come from the
steps (u = 2^-23, an ulp at most; a rounding is half of one):
  exp(x)          by the fast exponential, 2 + 1.173 |x| ulps, and what x itself
                  is off by times its size
  s = 1/(1 + e)   e's error times s (1 - s), and 3 ulps for sum and quotient
  Phi(z), z < 0   a product of the fit (8 ulps with its quotient) and exp(-z^2/2)
and first order error propagation from there."""
import math

import pytest
import torch

import ops_reference as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
u = 2.0 ** -23
A, B = 2 * math.sqrt(2 / math.pi), 0.044715


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_optimizer_device_gb300 as Z
    return Z


def every_bf16(lo, hi):
    bits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16)
    z = bits.view(BF)
    f = z.float()
    return z[(f >= lo) & (f <= hi) & ((f.abs() >= 2.0 ** -100) | (f == 0))]


def formulas(z, act):
    """act(z), act'(z) and what either may be off by, 64 bits."""
    z = z.to(R.D)
    if act == "gelu":
        phi = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        tail = torch.special.erfc(z.abs() / math.sqrt(2)) / 2
        s = torch.where(z < 0, tail, 1 - tail)
        rel = (z * z + 12) * u
        es = rel * tail + u * s
        return z * s, s + z * phi, z.abs() * es + u * (z * s).abs(), es + rel * (z * phi).abs() + u * (s + z * phi).abs()
    x, d, ex = (z, torch.ones_like(z), 0) if act == "silu" else \
        (A * (z + B * z ** 3), A + 3 * A * B * z * z, 2 * u)
    s = 1 / (1 + torch.exp(-x))
    t = 1 / (1 + torch.exp(x))
    es = s * t * ((2 + 1.173 * x.abs()) * u + ex * x.abs()) + 3 * u * s
    et = es + u * t
    v = z * s
    ev = z.abs() * es + u * v.abs()
    slope = s + v * t * d
    return v, slope, ev, es + d * (ev * t + v.abs() * et) + 4 * u * (s + (v * t * d).abs())


def values(Z, z, act, few):
    """act(z) in fp32: z as the inputs of a tile's rows, or as the weights of
    one token's outputs."""
    code = {"gelu": Z.ZERO_ACT_GELU, "gelu_tanh": Z.ZERO_ACT_GELU_TANH, "silu": Z.ZERO_ACT_SILU}[act]
    n = z.numel()
    col = torch.zeros(n, 8, dtype=BF, device="cuda")
    col[:, 0] = z.cuda()
    one = torch.ones(8, 8, dtype=BF, device="cuda")
    ep = Z.linear_epilogue(act=code)
    if few:
        y = torch.empty(1, n, device="cuda")
        Z.zero_linear(one, 8, col, 8, Z.ZERO_W_NK, 1, n, 1, ep, y, n, Z.ZERO_F32)
        return y[0].cpu()
    y = torch.empty(n, 8, device="cuda")
    Z.zero_linear(col, 8, one, 8, Z.ZERO_W_NK, n, 8, 1, ep, y, 8, Z.ZERO_F32)
    assert torch.equal(y[:, :1].expand_as(y).nan_to_num(7.0), y.nan_to_num(7.0))
    return y[:, 0].cpu()


def slopes(Z, z, act, rows):
    """act'(z) in fp32, z lying in `rows` rows."""
    code = {"gelu": Z.ZERO_ACT_GELU, "gelu_tanh": Z.ZERO_ACT_GELU_TANH, "silu": Z.ZERO_ACT_SILU}[act]
    k = -(-z.numel() // rows) + 7 & ~7
    pre = torch.zeros(rows, k, dtype=BF, device="cuda")
    pre.view(-1)[:z.numel()] = z.cuda()
    dy = torch.ones(rows, 8, dtype=BF, device="cuda")
    w = torch.ones(8, k, dtype=BF, device="cuda")
    dx = torch.empty(rows, k, device="cuda")
    Z.zero_linear_dinput(dy, 8, w, k, Z.ZERO_W_NK, rows, 1, k, Z.linear_act_grad(code, pre, k), dx, k,
                         Z.ZERO_F32)
    return dx.view(-1)[:z.numel()].cpu()


def check(z, got, want, err, what):
    bad = ~((got.to(R.D) - want).abs() <= err + 1e-37)
    if bad.any():
        i = int(bad.nonzero()[0])
        off = ((got.to(R.D) - want).abs() / want.abs().clamp_min(1e-300))[bad].max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, by up to {off:.3g} of "
                             f"themselves, first {z[i].item()}: {got[i]:.9g} for {want[i]:.9g}")


RANGES = [("gelu", -12.5), ("gelu_tanh", -9.0), ("silu", -80.0)]


@pytest.mark.parametrize("few", [True, False], ids=["one token", "tiles"])
@pytest.mark.parametrize("act,lo", RANGES)
def test_values_in_relative_terms(cuda, Z, act, lo, few):
    z = every_bf16(lo, 100.0)
    v, _, ev, _ = formulas(z, act)
    check(z, values(Z, z, act, few), v, ev, act)


@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("act,lo", RANGES)
def test_slopes_in_relative_terms(cuda, Z, act, lo, rows):
    z = every_bf16(lo, 100.0)
    _, s, _, es = formulas(z, act)
    check(z, slopes(Z, z, act, rows), s, es, act + "'")


@pytest.mark.parametrize("act", [a for a, _ in RANGES])
def test_values_and_slopes_of_huge_inputs(cuda, Z, act):
    """Up to bf16's largest finite value: z itself and a slope of 1 on one
    side, 0 and 0 on the other."""
    z = torch.cat([every_bf16(-3.4e38, -200.0), every_bf16(200.0, 3.4e38)])
    up = (z > 0).float()
    for few in (True, False):
        assert torch.equal(values(Z, z, act, few).abs(), z.float() * up)
    for rows in (1, 300):
        assert torch.equal(slopes(Z, z, act, rows).abs(), up)
