"""4-bit matrices and their products on the GPU against their definition in 64
bits: codes and scales byte for byte, products within the bounds that
ops_reference derives for sums in fp32, on what the codes stand for."""
import math

import pytest
import torch

import fp4_reference as Q
import ops_reference as R
from test_gpu_ops import Guarded, acts, code, randn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_optimizer_device_gb300 as Z
    return Z


def fmt(Z, form):
    return Z.ZERO_FP4_NV if form == "nv" else Z.ZERO_FP4_MX


class Packed:
    """A 4-bit matrix's buffers between canaries, rows `pad` bytes longer than they fill."""

    def __init__(self, Z, rows, cols, form, pad=0, g=None):
        self.rows, self.cols, self.form = rows, cols, form
        self.row, self.size = Z.zero_fp4_size(rows, cols, fmt(Z, form))
        assert (self.row, self.size) == Q.size(rows, cols, form)
        self.ld = self.row + pad
        self.codes_buf = torch.full((64 + rows * self.ld + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        self.codes = self.codes_buf.as_strided((rows, self.row), (self.ld, 1), 64)
        self.scales_buf = torch.full((64 + self.size + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        self.scales = self.scales_buf[64:64 + self.size]
        self.g = g
        self.mat = Z.fp4_matrix(self.codes, self.ld, self.scales, g)

    def fill(self, code_, byte):
        c, s = Q.pack(code_, byte, self.form)
        self.codes.copy_(c)
        self.scales.copy_(s)
        return self

    def check(self, code_, byte, what):
        c, s = Q.pack(code_, byte, self.form)
        got = self.codes.cpu()
        for lo in (0, 4):       # the sign of a zero does not matter
            a, b = (got >> lo) & 15, (c >> lo) & 15
            same = (a == b) | ((a & 7) + (b & 7) == 0)
            assert bool(same.all()), f"{what}: codes differ at {(~same).nonzero()[:3].tolist()}"
        assert torch.equal(self.scales.cpu(), s), f"{what}: scales differ at {(self.scales.cpu() != s).nonzero()[:5].flatten().tolist()}"
        left = self.codes_buf.clone()
        left.as_strided((self.rows, self.row), (self.ld, 1), 64).fill_(0xA5)
        assert bool((left == 0xA5).all()), f"{what}: wrote outside the codes"
        assert bool((self.scales_buf[:64] == 0xA5).all() and (self.scales_buf[64 + self.size:] == 0xA5).all()), f"{what}: wrote outside the scales"


def hard_values(g, rows, cols, dtype):
    """Normal values among blocks of other sizes, exact ties, zeros and the ends of the range."""
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-12, 12, (rows, 1), generator=g).float())
    x = x * torch.randn(cols, generator=g).mul(1.5).exp()
    pick = torch.rand(rows, cols, generator=g)
    tie = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.0])
    x = torch.where(pick < 0.05, tie[torch.randint(0, 9, (rows, cols), generator=g)], x)
    x = torch.where(pick > 0.97, torch.zeros(()), x)
    return x.to(dtype)


SHAPES = [(1, 1), (1, 16), (1, 33), (3, 15), (2, 17), (5, 70), (17, 31), (33, 100), (128, 128), (129, 64), (127, 257), (300, 520), (1, 4096), (1000, 3)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", ["mx", "nv"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_and_back(cuda, Z, rows, cols, form, dtype):
    g = torch.Generator().manual_seed(rows * 1009 + cols)
    x = hard_values(g, rows, cols, dtype)
    for pad, skew, extra in ((0, 0, 0), (3, 1, 16), (8, 0, 64)):
        X = Guarded(rows, cols, dtype, pad, skew, x)
        scale = torch.full((1,), -1.0, device="cuda") if form == "nv" else None
        if scale is not None:
            work = torch.empty(Z.ZERO_FP4_WORKSPACE, dtype=torch.uint8, device="cuda")
            Z.zero_fp4_tensor_scale(X.t, X.ld, code(Z, dtype), rows, cols, scale, work, work.numel())
            assert scale.item() == Q.tensor_scale(x).item()
        ref, ref_t = (Q.quantise(v, form, None if scale is None else Q.tensor_scale(x)) for v in (x, x.t()))
        q, qt = Packed(Z, rows, cols, form, extra, scale), Packed(Z, cols, rows, form, extra, scale)
        Z.zero_fp4_quantize(X.t, X.ld, code(Z, dtype), rows, cols, fmt(Z, form), q.mat, qt.mat)
        q.check(*ref[:2], "q")
        qt.check(*ref_t[:2], "qt")
        for one, alone in ((0, Packed(Z, rows, cols, form, extra, scale)), (1, Packed(Z, cols, rows, form, extra, scale))):
            Z.zero_fp4_quantize(X.t, X.ld, code(Z, dtype), rows, cols, fmt(Z, form), None if one else alone.mat, alone.mat if one else None)
            alone.check(*(ref_t if one else ref)[:2], "alone")
        for out in (BF, F32):
            Y = Guarded(rows, cols, out, pad, skew)
            Z.zero_fp4_dequantize(q.mat, rows, cols, fmt(Z, form), Y.t, Y.ld, code(Z, out))
            assert torch.equal(Y.t.cpu(), ref[2].to(F32).to(out))
            Y.check("y")


@pytest.mark.parametrize("form", ["mx", "nv"])
def test_quantize_what_is_not_finite_and_the_ends_of_the_range(cuda, Z, form):
    """A NaN or an infinity takes its own block alone; subnormals and the largest values keep to the definition."""
    x = torch.randn(64, 256, generator=torch.Generator().manual_seed(1))
    x[0, 0], x[1, 17], x[2, 40], x[63, 255] = float("nan"), float("inf"), -float("inf"), float("nan")
    x[5], x[6], x[7], x[8] = 0.0, 1e-40, 3e38, -1.17e-38
    x[9, :32] = torch.linspace(-6, 6, 32)
    for dtype in (BF, F32):
        v = x.to(dtype)
        scale = None if form == "mx" else torch.full((1,), 0.01, device="cuda")
        g = None if form == "mx" else torch.tensor(0.01, dtype=F32)
        X = v.cuda()
        q, qt = Packed(Z, 64, 256, form, 0, scale), Packed(Z, 256, 64, form, 0, scale)
        Z.zero_fp4_quantize(X, 256, code(Z, dtype), 64, 256, fmt(Z, form), q.mat, qt.mat)
        ref, ref_t = Q.quantise(v, form, g), Q.quantise(v.t(), form, g)
        q.check(*ref[:2], "q")
        qt.check(*ref_t[:2], "qt")
        y = torch.empty(64, 256, device="cuda")
        Z.zero_fp4_dequantize(q.mat, 64, 256, fmt(Z, form), y, 256, Z.ZERO_F32)
        assert torch.equal(torch.nan_to_num(y.cpu(), nan=-7.0), torch.nan_to_num(ref[2].to(F32), nan=-7.0))


@pytest.mark.parametrize("values,want", [([0.0] * 40, 1.0), ([float("nan"), float("inf")] * 20, 1.0), ([-5376.0, float("-inf")] + [1.0] * 38, 2.0)])
def test_tensor_scale_of_zeros_and_infinities(cuda, Z, values, want):
    x, g = torch.tensor([values], device="cuda"), torch.zeros(1, device="cuda")
    work = torch.empty(Z.ZERO_FP4_WORKSPACE, dtype=torch.uint8, device="cuda")
    Z.zero_fp4_tensor_scale(x, 40, Z.ZERO_F32, 1, 40, g, work, work.numel())
    assert g.item() == want
    g.fill_(-1)
    Z.zero_fp4_tensor_scale(x, 40, Z.ZERO_F32, 0, 40, g, work, work.numel())
    assert g.item() == 1.0


@pytest.mark.parametrize("form", ["mx", "nv"])
def test_nothing_to_quantize(cuda, Z, form):
    for rows, cols in ((0, 8), (8, 0)):
        q, qt = Packed(Z, 8, 8, form), Packed(Z, 8, 8, form)
        x = torch.ones(8, 8, device="cuda")
        Z.zero_fp4_quantize(x, 8, Z.ZERO_F32, rows, cols, fmt(Z, form), q.mat, qt.mat)
        y = Guarded(8, 8, F32)
        Z.zero_fp4_dequantize(q.mat, rows, cols, fmt(Z, form), y.t, 8, Z.ZERO_F32)
        torch.cuda.synchronize()
        for b in (q.codes_buf, q.scales_buf, qt.codes_buf, qt.scales_buf):
            assert bool((b == 0xA5).all())
        assert bool((y.buf == -77.0).all())


def operand(Z, g, rows, cols, form, pad=0, scale=1.0):
    """A random 4-bit operand, and in doubles what it stands for without g, and g."""
    x = torch.randn(rows, cols, generator=g) * scale
    whole = None
    if form == "nv":
        whole = Q.tensor_scale(x)
    c, b, v = Q.quantise(x, form, whole)
    dev = None if whole is None else whole.to(F32).reshape(1).cuda()
    unit = Q.LEVELS[(c & 7).long()] * torch.where(c > 7, -1.0, 1.0)
    s = Q.E4M3[b.long()] if form == "nv" else torch.ldexp(torch.ones(b.shape, dtype=Q.D), b.int() - 127)
    unit = unit * s.repeat_interleave(Q.SIZE[form], 1)[:, :cols]
    return Packed(Z, rows, cols, form, pad, dev).fill(c, b), unit, 1.0 if whole is None else whole.item()


def run_linear(Z, m, n, k, form, *, seed=0, bias=None, act="none", pre=False, gate=False, p=None, residual=None, out=BF, pad=0, skew=0, in_place=False):
    g = torch.Generator().manual_seed(seed * 7919 + m * 31 + n * 17 + k)
    x, vx, gx = operand(Z, g, m, k, form, 16 * (pad % 3))
    w, vw, gw = operand(Z, g, n, k, form, 0, 1 / math.sqrt(max(k, 1)))
    vw = vw * (gx * gw)
    b = None if bias is None else randn(g, n, dtype=bias)
    u = randn(g, m, n) if gate else None
    r = None if residual is None else randn(g, m, n, dtype=residual)
    U = Guarded(m, n, BF, pad, skew, u) if gate else None
    Y = Guarded(m, n, out, pad, skew, r if in_place else None)
    Rs = Y if in_place else (Guarded(m, n, residual, pad, skew, r) if residual is not None else None)
    P = Guarded(m, n, BF, pad, skew) if pre else None
    Bv = None if b is None else Guarded(1, n, b.dtype, 0, skew, b[None])
    rng = None if p is None else Z.dropout_rng(p, 0x1234567890ABCDEF, 99 + seed)
    ep = Z.linear_epilogue(bias=None if Bv is None else Bv.t[0], bias_dtype=code(Z, bias), act=acts(Z)[act], pre=P.t if pre else None,
                           ldpre=P.ld if pre else 0, gate=U.t if gate else None, ldgate=U.ld if gate else 0, residual=Rs.t if Rs else None,
                           ldres=Rs.ld if Rs else 0, res_dtype=code(Z, residual), dropout=rng)
    Z.zero_fp4_linear(x.mat, w.mat, fmt(Z, form), m, n, k, ep, Y.t, Y.ld, code(Z, out))
    torch.cuda.synchronize()
    y, z, ey, ez = R.linear(vx, vw, False, b, act, u, p, 0x1234567890ABCDEF, 99 + seed, r)
    R.assert_within(Y.t, y, ey, "y")
    Y.check("y")
    if pre:
        R.assert_within(P.t, z, ez, "pre")
        P.check("pre")


SIZES = [(1, 8, 32), (1, 1, 1), (1, 257, 1031), (3, 130, 64), (16, 256, 512), (33, 64, 2048), (100, 129, 65), (127, 127, 127), (128, 128, 256), (129, 256, 192),
         (130, 384, 128), (200, 192, 300), (256, 576, 256), (300, 520, 331), (512, 264, 1000), (1000, 777, 40), (77, 2304, 768)]


@pytest.mark.parametrize("form", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_plain(cuda, Z, m, n, k, form):
    run_linear(Z, m, n, k, form)
    run_linear(Z, m, n, k, form, out=F32, bias=F32, seed=1)


@pytest.mark.parametrize("form", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", [(1, 96, 64), (7, 130, 72), (130, 258, 136), (200, 99, 33), (520, 768, 768), (300, 200, 1030)])
def test_linear_everything(cuda, Z, m, n, k, form):
    run_linear(Z, m, n, k, form, bias=BF, act="gelu_tanh", pre=True, gate=True, p=0.1, residual=BF)
    run_linear(Z, m, n, k, form, bias=F32, act="silu", pre=True, gate=True, p=0.5, residual=F32, out=F32, pad=8)
    run_linear(Z, m, n, k, form, act="relu", residual=BF, p=0.25, in_place=True, pad=1, skew=3)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_linear_activations(cuda, Z, act, out):
    run_linear(Z, 140, 200, 96, "nv", act=act, out=out)


@pytest.mark.parametrize("form", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k,pad", [(2100, 2500, 72, 0), (2100, 2500, 840, 4), (2050, 2563, 90, 0), (2100, 3500, 5000, 0)])
def test_more_tiles_than_the_gpu_holds(cuda, Z, m, n, k, pad, form):
    """Several tiles per pair of CTAs, the last ragged both ways; fp32 rounds."""
    run_linear(Z, m, n, k, form, bias=BF, act="gelu_tanh", pre=True, gate=True, residual=BF, pad=pad)
    run_linear(Z, m, n, k, form, bias=F32, act="silu", residual=F32, out=F32, pad=pad)


@pytest.mark.parametrize("form", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", [(1, 40, 70), (5, 260, 130), (65, 96, 1000), (140, 300, 264), (520, 200, 768), (1000, 1030, 90)])
def test_dinput(cuda, Z, m, n, k, form):
    for act, gate, out, pad, skew in ((None, False, BF, 0, 0), (None, False, F32, 0, 0), ("gelu_tanh", False, BF, 0, 0), ("silu", True, BF, 8, 0),
                                      ("relu", True, F32, 1, 1)):
        g = torch.Generator().manual_seed(m + 3 * n + 5 * k)
        dy, vd, gd = operand(Z, g, m, n, form)
        w, vw, gw = operand(Z, g, k, n, form, 16, 1 / math.sqrt(n))
        pre, u = randn(g, m, k), randn(g, m, k)
        P, U = Guarded(m, k, BF, pad, skew, pre), Guarded(m, k, BF, pad, skew, u)
        DX, DU = Guarded(m, k, out, pad, skew), Guarded(m, k, BF, pad, skew)
        ag = None
        if act is not None:
            ag = Z.linear_act_grad(acts(Z)[act], P.t, P.ld, U.t if gate else None, U.ld if gate else 0, DU.t if gate else None, DU.ld if gate else 0)
        Z.zero_fp4_linear_dinput(dy.mat, w.mat, fmt(Z, form), m, n, k, ag, DX.t, DX.ld, code(Z, out))
        torch.cuda.synchronize()
        dx, du, ex, eu = R.linear_dinput(vd, vw * (gd * gw), True, act, pre, u if gate else None)
        R.assert_within(DX.t, dx, ex, "dx")
        DX.check("dx")
        if gate:
            R.assert_within(DU.t, du, eu, "dgate")
            DU.check("dgate")


@pytest.mark.parametrize("form", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", [(1, 40, 70), (64, 260, 130), (1000, 96, 65), (333, 300, 264), (40, 1000, 520), (5000, 300, 200)])
def test_dweight(cuda, Z, m, n, k, form):
    for out, add, pad, skew in ((BF, False, 0, 0), (F32, True, 0, 0), (BF, True, 8, 0), (F32, False, 1, 3), (F32, True, 5, 1)):
        g = torch.Generator().manual_seed(m + 3 * n + 5 * k)
        dy, vd, gd = operand(Z, g, n, m, form)
        x, vx, gx = operand(Z, g, k, m, form, 32)
        old = randn(g, n, k, dtype=out)
        DW = Guarded(n, k, out, pad, skew, old)
        Z.zero_fp4_linear_dweight(dy.mat, x.mat, fmt(Z, form), m, n, k, DW.t, DW.ld, code(Z, out), add)
        torch.cuda.synchronize()
        dw, _, ew, _ = R.linear_dweight(vd.T, vx.T * (gd * gx), False, old if add else None)
        R.assert_within(DW.t, dw, ew, "dw")
        DW.check("dw")


def test_nothing_to_multiply(cuda, Z):
    """k = 0: the epilogue of the bias alone; m or n = 0: nothing is written."""
    run_linear(Z, 9, 40, 0, "mx", bias=BF, act="silu")
    run_linear(Z, 200, 300, 0, "nv")
    q = Packed(Z, 8, 32, "mx").fill(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 1, dtype=torch.uint8))
    for m, n in ((0, 8), (8, 0)):
        Y = Guarded(8, 8, BF)
        Z.zero_fp4_linear(q.mat, q.mat, Z.ZERO_FP4_MX, m, n, 32, None, Y.t, 8)
        torch.cuda.synchronize()
        assert bool((Y.buf == -77.0).all())


@pytest.mark.parametrize("form", ["mx", "nv"])
def test_a_block_of_nan_reaches_its_own_row_alone(cuda, Z, form):
    for m, n, k in ((64, 200, 96), (300, 260, 600)):
        x, w = torch.randn(m, k).to(BF), torch.randn(n, k).to(BF)
        x[3, 5], w[7, k - 1] = float("inf"), float("nan")
        X, W = x.cuda(), w.cuda()
        ones = None if form == "mx" else torch.ones(1, device="cuda")
        qx, qw = Packed(Z, m, k, form, 0, ones), Packed(Z, n, k, form, 0, ones)
        Z.zero_fp4_quantize(X, k, Z.ZERO_BF16, m, k, fmt(Z, form), qx.mat)
        Z.zero_fp4_quantize(W, k, Z.ZERO_BF16, n, k, fmt(Z, form), qw.mat)
        y = torch.empty(m, n, device="cuda")
        Z.zero_fp4_linear(qx.mat, qw.mat, fmt(Z, form), m, n, k, None, y, n, Z.ZERO_F32)
        bad = torch.isnan(y.cpu())
        want = torch.zeros(m, n, dtype=torch.bool)
        want[3], want[:, 7] = True, True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("m,n,k", [(16, 96, 36000), (300, 264, 36000), (700, 2048, 32768)])
def test_fp32_results_of_long_sums(cuda, Z, m, n, k):
    """As for bf16 products: 48 truncating additions a round, each half a unit
    in the last place of the running sum on average: 48 * 2^-24 = 2.9e-6."""
    g = torch.Generator().manual_seed(6)
    x, vx, gx = operand(Z, g, m, k, "nv")
    w, vw, gw = operand(Z, g, n, k, "nv")
    y = torch.empty(m, n, device="cuda")
    Z.zero_fp4_linear(x.mat, w.mat, Z.ZERO_FP4_NV, m, n, k, None, y, n, Z.ZERO_F32)
    want = (vx.cuda() @ vw.cuda().T) * (gx * gw)
    assert ((y.double() - want).norm() / want.norm()).item() < 2.9e-6
