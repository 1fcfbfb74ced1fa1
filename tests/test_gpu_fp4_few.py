"""4-bit products of one to eight rows on both of their paths: weights so wide
that tiles take them, and contractions that go round the copies' ring."""
import math

import pytest
import torch

import ops_reference as R
from test_gpu_fp4 import fmt, operand, run_linear
from test_gpu_ops import Guarded, acts, code, randn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_optimizer_device_gb300 as Z
    return Z


@pytest.mark.parametrize("form", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", [(1, 16411, 512), (8, 17000, 600), (3, 33001, 72), (8, 40, 20000), (1, 130, 33000), (5, 1030, 8200)])
def test_wide_and_deep(cuda, Z, m, n, k, form):
    run_linear(Z, m, n, k, form)
    run_linear(Z, m, n, k, form, bias=BF, act="silu", pre=True, gate=True, p=0.2, residual=F32, out=F32, pad=3, seed=2)


@pytest.mark.parametrize("form", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", [(1, 500, 17003), (8, 72, 20000), (4, 9000, 60)])
def test_dinput_wide_and_deep(cuda, Z, m, n, k, form):
    g = torch.Generator().manual_seed(m + 3 * n + 5 * k)
    dy, vd, gd = operand(Z, g, m, n, form)
    w, vw, gw = operand(Z, g, k, n, form, 16, 1 / math.sqrt(n))
    pre, u = randn(g, m, k), randn(g, m, k)
    P, U, DX, DU = Guarded(m, k, BF, 8, 0, pre), Guarded(m, k, BF, 8, 0, u), Guarded(m, k, BF, 8, 0), Guarded(m, k, BF, 8, 0)
    ag = Z.linear_act_grad(acts(Z)["silu"], P.t, P.ld, U.t, U.ld, DU.t, DU.ld)
    Z.zero_fp4_linear_dinput(dy.mat, w.mat, fmt(Z, form), m, n, k, ag, DX.t, DX.ld, code(Z, BF))
    torch.cuda.synchronize()
    dx, du, ex, eu = R.linear_dinput(vd, vw * (gd * gw), True, "silu", pre, u)
    R.assert_within(DX.t, dx, ex, "dx")
    R.assert_within(DU.t, du, eu, "dgate")
    DX.check("dx")
    DU.check("dgate")


@pytest.mark.parametrize("form", ["mx", "nv"])
def test_rows_do_not_depend_on_their_neighbours(cuda, Z, form):
    """A row's result is the same, bit for bit, whichever rows stand beside it and
    whenever it is computed."""
    n, k = 264, 9000
    g = torch.Generator().manual_seed(5)
    w, _, _ = operand(Z, g, n, k, form)
    x, _, _ = operand(Z, g, 8, k, form)
    y = torch.empty(8, n, device="cuda")
    Z.zero_fp4_linear(x.mat, w.mat, fmt(Z, form), 8, n, k, None, y, n, Z.ZERO_F32)
    for m in (1, 3, 8):
        z = torch.empty(m, n, device="cuda")
        Z.zero_fp4_linear(x.mat, w.mat, fmt(Z, form), m, n, k, None, z, n, Z.ZERO_F32)
        assert torch.equal(z, y[:m])


@pytest.mark.parametrize("form", ["mx", "nv"])
def test_nothing_to_contract(cuda, Z, form):
    """k = 0: the bias alone through the epilogue."""
    run_linear(Z, 3, 40, 0, form, bias=BF, act="silu", residual=F32)


@pytest.mark.parametrize("form", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", [(700, 1, 40), (700, 8, 130), (4100, 5, 264), (90, 3, 20000)])
def test_dweight_of_few_outputs(cuda, Z, m, n, k, form):
    for out, add in ((F32, True), (BF, False), (BF, True)):
        g = torch.Generator().manual_seed(m + 3 * n + 5 * k)
        dy, vd, gd = operand(Z, g, n, m, form)
        x, vx, gx = operand(Z, g, k, m, form, 32)
        old = randn(g, n, k, dtype=out)
        DW = Guarded(n, k, out, 5, 1, old)
        Z.zero_fp4_linear_dweight(dy.mat, x.mat, fmt(Z, form), m, n, k, DW.t, DW.ld, code(Z, out), add)
        torch.cuda.synchronize()
        dw, _, ew, _ = R.linear_dweight(vd.T, vx.T * (gd * gx), False, old if add else None)
        R.assert_within(DW.t, dw, ew, "dw")
        DW.check("dw")
