"""Llama's gated feed-forward sublayer as a whole, forward and backward, against
64-bit autograd of its formulas; and matrices whose rows lie so far apart that
offsets pass 2^31 elements."""
import pytest
import torch

import ops_reference as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_optimizer_device_gb300 as Z
    return Z


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,d,f", [(1, 32, 88), (77, 64, 176), (300, 96, 264), (260, 50, 130)])
def test_gated_sublayer_against_autograd(cuda, Z, m, d, f, wide):
    """y = h + (silu(u Wg') * (u Wu')) Wd', u = RMS norm of h.  The input's
    gradient is a sum of two products: zero_linear_dinput for one branch, and
    zero_linear with the weight in its other layout and that as its residual,
    in place, for the other."""
    g = torch.Generator().manual_seed(m + f)
    rn = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(BF)  # noqa: E731
    h, dy = rn(m, d), rn(m, d)
    nw, wg, wu, wd = (rn(d, scale=0.1).float() + 1).to(BF), rn(f, d, scale=d ** -0.5), rn(f, d, scale=d ** -0.5), \
        rn(d, f, scale=f ** -0.5)
    H, DY, NW, WG, WU, WD = (t.cuda() for t in (h, dy, nw, wg, wu, wd))
    new = lambda *s, t=BF: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    u, up, z, a, y, dz, dup, dh = new(m, d), new(m, f), new(m, f), new(m, f), new(m, d), new(m, f), new(m, f), new(m, d)
    dwg, dwu, dwd, dnw, rstd = new(f, d), new(f, d), new(d, f), new(d), new(m, t=F32)
    nk, kn, bf = Z.ZERO_W_NK, Z.ZERO_W_KN, Z.ZERO_BF16
    Z.zero_layer_norm(H, d, bf, NW, None, bf, m, d, Z.ZERO_NORM_RMS, 1e-5, u, d, bf, None, rstd)
    Z.zero_linear(u, d, WU, d, nk, m, f, d, None, up, f)
    Z.zero_linear(u, d, WG, d, nk, m, f, d,
                  Z.linear_epilogue(act=Z.ZERO_ACT_SILU, pre=z, ldpre=f, gate=up, ldgate=f), a, f)
    Z.zero_linear(a, f, WD, f, nk, m, d, f, Z.linear_epilogue(residual=H, ldres=d), y, d)
    Z.zero_linear_dweight(DY, d, a, f, m, d, f, nk, dwd, f)
    Z.zero_linear_dinput(DY, d, WD, f, nk, m, d, f,
                         Z.linear_act_grad(Z.ZERO_ACT_SILU, z, f, up, f, dup, f), dz, f)
    Z.zero_linear_dweight(dz, f, u, d, m, f, d, nk, dwg, d)
    Z.zero_linear_dweight(dup, f, u, d, m, f, d, nk, dwu, d)
    dt = Z.ZERO_F32 if wide else bf
    du = new(m, d, t=F32 if wide else BF)
    Z.zero_linear_dinput(dz, f, WG, d, nk, m, f, d, None, du, d, dt)
    Z.zero_linear(dup, f, WU, d, kn, m, d, f, Z.linear_epilogue(residual=du, ldres=d, res_dtype=dt), du, d, dt)
    size = Z.zero_layer_norm_workspace(m, d)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    Z.zero_layer_norm_backward(du, d, dt, H, d, bf, NW, bf, None, rstd, m, d, Z.ZERO_NORM_RMS, DY, d, dh, d, bf,
                               dnw, None, bf, False, work, size)

    D = R.D
    p = [t.to(D).requires_grad_() for t in (h, nw, wg, wu, wd)]
    hd, nwd, wgd, wud, wdd = p
    ud = hd * (hd.square().mean(1, keepdim=True) + 1e-5).rsqrt() * nwd
    zd = ud @ wgd.T
    want = hd + (zd * torch.sigmoid(zd) * (ud @ wud.T)) @ wdd.T
    want.backward(dy.to(D))
    # at most eight bf16 roundings lie between the inputs and the furthest
    # gradient, each 2^-9 of a value in the mean; products average them
    rel = lambda x, w: ((x.cpu().to(D) - w).norm() / w.norm()).item()  # noqa: E731
    for name, got, ref in (("y", y, want.detach()), ("dh", dh, hd.grad), ("dnorm", dnw, nwd.grad),
                           ("dgate weight", dwg, wgd.grad), ("dup weight", dwu, wud.grad),
                           ("ddown weight", dwd, wdd.grad)):
        assert rel(got, ref) < 8 * 2.0 ** -8, name


FAR = 1 << 27        # elements between rows; 20 rows reach beyond 2^31


def far(m, n, ld, fill=None):
    t = torch.empty((m - 1) * ld + n, dtype=BF, device="cuda").as_strided((m, n), (ld, 1))
    if fill is not None:
        t.copy_(fill)
    return t


@pytest.mark.parametrize("odd", [0, 3], ids=["aligned", "odd"])
@pytest.mark.parametrize("m", [20, 150])
def test_rows_far_apart(cuda, Z, m, odd):
    """Offsets beyond 2^31 elements in inputs and outputs of every operator."""
    ld = (FAR if m == 20 else FAR >> 2) + 8 + odd
    assert (m - 1) * ld > 1 << 31
    g = torch.Generator().manual_seed(m)
    n, k = 72, 104
    rn = lambda *s: torch.randn(*s, generator=g).to(BF)  # noqa: E731
    x, w, r = rn(m, k), rn(n, k), rn(m, n)
    X, Y = far(m, k, ld, x), far(m, n, ld)
    W = w.cuda()
    Z.zero_linear(X, ld, W, k, Z.ZERO_W_NK, m, n, k, Z.linear_epilogue(residual=r.cuda(), ldres=n), Y, ld)
    y, _, ey, _ = R.linear(x, w, False, residual=r)
    R.assert_within(Y, y, ey, "y")
    Y.copy_(r)                                   # now the gradient
    DW = torch.empty(n, k, device="cuda")
    Z.zero_linear_dweight(Y, ld, X, ld, m, n, k, Z.ZERO_W_NK, DW, k, Z.ZERO_F32)
    dw, _, ew, _ = R.linear_dweight(r, x, False)
    R.assert_within(DW, dw, ew, "dw")
    Z.zero_linear_dinput(Y, ld, W, k, Z.ZERO_W_NK, m, n, k, None, X, ld)
    dx, _, ex, _ = R.linear_dinput(r, w, False)
    R.assert_within(X, dx, ex, "dx")
    X.copy_(x)
    Z.zero_dropout(X, ld, 1, None, 0, 1, m, k, Z.dropout_rng(0.25, 3, 4), X, ld, 1)
    want = R.drop(x.to(R.D), 0.25, 3, 4)
    R.assert_within(X, want, 4 * R.U32 * want.abs(), "dropout")
    X.copy_(x)
    nw = rn(k)
    rstd = torch.empty(m, device="cuda")
    D = torch.empty(m, k, dtype=BF, device="cuda")
    Z.zero_layer_norm(X, ld, 1, nw.cuda(), None, 1, m, k, Z.ZERO_NORM_RMS, 1e-5, D, k, 1, None, rstd)
    v, _, rs, ev = R.norm(x, nw, None, True, 1e-5)
    R.assert_within(D, v, ev, "norm")
    dy = rn(m, k)
    size = Z.zero_layer_norm_workspace(m, k)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    dnw = torch.empty(k, device="cuda")
    Z.zero_layer_norm_backward(dy.cuda(), k, 1, X, ld, 1, nw.cuda(), 1, None, rstd, m, k, Z.ZERO_NORM_RMS, None, 0,
                               D, k, 1, dnw, None, 0, False, work, size)
    dx, dw, _, ex, ew, _ = R.norm_backward(dy, x, nw, None, rstd.cpu(), True)
    R.assert_within(D, dx, ex, "norm dx")
    R.assert_within(dnw, dw, ew, "norm dw")
