"""The layer operators on the GPU against their formulas in 64 bits, at the
sizes, strides and values where they can go wrong.  Every bound is derived in
ops_reference from the number of fp32 operations and one rounding of the
output; outputs lie between guard bands that must stay untouched."""
import math

import pytest
import torch

import ops_reference as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
GUARD = 64


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_optimizer_device_gb300 as Z
    return Z


def code(Z, dtype):
    return Z.ZERO_F32 if dtype == F32 else Z.ZERO_BF16


def acts(Z):
    return dict(zip(R.ACTS, (Z.ZERO_ACT_NONE, Z.ZERO_ACT_RELU, Z.ZERO_ACT_GELU,
                             Z.ZERO_ACT_GELU_TANH, Z.ZERO_ACT_SILU)))


class Guarded:
    """An [m, n] matrix (rows ld apart, `skew` elements off a 256-byte
    boundary) inside a buffer of canaries: the gaps between rows and both ends
    must keep them."""

    def __init__(self, m, n, dtype, pad=0, skew=0, fill=None):
        self.m, self.n, self.ld = m, n, n + pad
        size = GUARD + skew + m * self.ld + GUARD
        self.buf = torch.full((size,), -77.0, dtype=dtype, device="cuda")
        self.t = self.buf.as_strided((m, n), (self.ld, 1), GUARD + skew)
        if fill is not None:
            self.t.copy_(fill)

    def check(self, what):
        b = self.buf.clone()
        b.as_strided((self.m, self.n), (self.ld, 1), self.t.storage_offset()).fill_(-77.0)
        assert bool((b == -77.0).all()), f"{what}: wrote outside the matrix"


def randn(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def cpu(t):
    return t.detach().cpu()


SIZES = [  # m, n, k: one token, few, tile edges on each side, odd, long sums
    (1, 8, 8), (1, 768, 768), (1, 1, 1), (1, 257, 1031), (3, 130, 64), (5, 127, 100),
    (16, 256, 512), (17, 136, 72), (33, 64, 2048), (64, 200, 4096), (100, 129, 65),
    (127, 127, 127), (128, 128, 64), (129, 256, 192), (130, 384, 128), (255, 1000, 96),
    (256, 256, 256), (300, 520, 331), (512, 264, 1000), (1000, 777, 40), (77, 2304, 768)]


def run_linear(Z, m, n, k, kn, *, seed=0, bias=None, act="none", pre=False, gate=False, p=None,
               residual=None, out=BF, pad=0, skew=0, in_place=False):
    g = torch.Generator().manual_seed(seed * 7919 + m * 31 + n * 17 + k)
    mk = lambda rows, cols, t: Guarded(rows, cols, t.dtype, pad, skew, t)  # noqa: E731
    x, w = randn(g, m, k), randn(g, *((k, n) if kn else (n, k)), scale=1 / math.sqrt(max(k, 1)))
    b = None if bias is None else randn(g, n, dtype=bias)
    u = randn(g, m, n) if gate else None
    r = None if residual is None else randn(g, m, n, dtype=residual)
    X, W = mk(m, k, x), mk(w.shape[0], w.shape[1], w)
    U = mk(m, n, u) if gate else None
    Y = Guarded(m, n, out, pad, skew, r if in_place else None)
    Rs = Y if in_place else (mk(m, n, r) if residual is not None else None)
    P = Guarded(m, n, BF, pad, skew) if pre else None
    Bv = None
    if b is not None:
        Bv = Guarded(1, n, b.dtype, 0, skew, b[None])
    rng = None if p is None else Z.dropout_rng(p, 0x1234567890ABCDEF, 99 + seed)
    ep = Z.linear_epilogue(
        bias=None if Bv is None else Bv.t[0], bias_dtype=code(Z, bias), act=acts(Z)[act],
        pre=P.t if pre else None, ldpre=P.ld if pre else 0,
        gate=U.t if gate else None, ldgate=U.ld if gate else 0,
        residual=Rs.t if Rs else None, ldres=Rs.ld if Rs else 0,
        res_dtype=code(Z, residual), dropout=rng)
    Z.zero_linear(X.t, X.ld, W.t, W.ld, Z.ZERO_W_KN if kn else Z.ZERO_W_NK, m, n, k, ep, Y.t, Y.ld,
                  code(Z, out))
    torch.cuda.synchronize()
    y, z, ey, ez = R.linear(x, w, kn, b, act, u, p, 0x1234567890ABCDEF, 99 + seed, r)
    R.assert_within(Y.t, y, ey, "y")
    Y.check("y")
    if pre:
        R.assert_within(P.t, z, ez, "pre")
        P.check("pre")
    return cpu(Y.t)


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_plain(cuda, Z, m, n, k, kn):
    run_linear(Z, m, n, k, kn)
    run_linear(Z, m, n, k, kn, out=F32, bias=F32, seed=1)


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("m,n,k", [(1, 96, 64), (7, 130, 72), (130, 258, 136), (200, 99, 33),
                                   (520, 768, 768)])
def test_linear_everything(cuda, Z, m, n, k, kn):
    run_linear(Z, m, n, k, kn, bias=BF, act="gelu_tanh", pre=True, gate=True, p=0.1, residual=BF)
    run_linear(Z, m, n, k, kn, bias=F32, act="silu", pre=True, gate=True, p=0.5, residual=F32,
               out=F32, pad=8)
    run_linear(Z, m, n, k, kn, act="relu", residual=BF, p=0.25, in_place=True)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_linear_activations(cuda, Z, act, out):
    run_linear(Z, 140, 200, 96, False, act=act, out=out)


@pytest.mark.parametrize("pad,skew", [(0, 0), (8, 0), (1, 3)])
@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("n,k", [(1, 4099), (31, 8), (260, 1000), (33, 264), (1000, 64), (520, 2056)])
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 9])
def test_few_rows(cuda, Z, m, n, k, kn, pad, skew):
    """Tokens being generated: every count of rows, outputs that end inside a
    warp's four and a block's 32, contractions of one piece and of many."""
    run_linear(Z, m, n, k, kn, bias=F32, act="silu", pre=True, gate=True, residual=BF, p=0.25,
               pad=pad, skew=skew)
    run_linear(Z, m, n, k, kn, out=F32, pad=pad, skew=skew)


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("m,n,k", [(1, 1000, 33), (3, 264, 512), (7, 129, 260), (8, 2056, 40)])
def test_few_rows_gradient(cuda, Z, m, n, k, kn):
    g = torch.Generator().manual_seed(m * n + k)
    dy, w = randn(g, m, n), randn(g, *((k, n) if kn else (n, k)), scale=n ** -0.5)
    pre, u = randn(g, m, k), randn(g, m, k)
    lay = Z.ZERO_W_KN if kn else Z.ZERO_W_NK
    DX, DU = Guarded(m, k, F32, 1), Guarded(m, k, BF, 3, 5)
    D, W, P, U = (t.cuda() for t in (dy, w, pre, u))
    ag = Z.linear_act_grad(Z.ZERO_ACT_GELU, P, k, U, k, DU.t, DU.ld)
    Z.zero_linear_dinput(D, n, W, W.shape[1], lay, m, n, k, ag, DX.t, DX.ld, Z.ZERO_F32)
    dx, du, ex, eu = R.linear_dinput(dy, w, kn, "gelu", pre, u)
    R.assert_within(DX.t, dx, ex, "dx")
    R.assert_within(DU.t, du, eu, "dgate")
    DX.check("dx")
    DU.check("dgate")


@pytest.mark.parametrize("pad,skew", [(1, 0), (0, 1), (3, 5), (8, 0), (4, 4), (2, 2), (8, 8)])
@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("m,n,k", [(1, 64, 200), (40, 96, 136), (300, 264, 200)])
def test_linear_strides_and_alignments(cuda, Z, m, n, k, kn, pad, skew):
    run_linear(Z, m, n, k, kn, bias=BF, act="gelu", pre=True, residual=F32, pad=pad, skew=skew)


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("m,n,k", [(300, 259, 331), (300, 256, 331), (600, 1001, 77), (90, 203, 131)])
def test_odd_sizes_in_aligned_rows(cuda, Z, m, n, k, kn):
    """Odd sizes whose rows are padded to 16 bytes: what lies in the gaps
    (-77) enters no sum, and no store reaches into them."""
    g = torch.Generator().manual_seed(m + n + k)

    def mk(t):
        rows, cols = t.shape
        return Guarded(rows, cols, t.dtype, -cols % 8, 0, t)

    x, w = randn(g, m, k), randn(g, *((k, n) if kn else (n, k)), scale=k ** -0.5)
    r, dy, pre, u = randn(g, m, n), randn(g, m, n), randn(g, m, k), randn(g, m, k)
    X, W, Q, DY, P, U = (mk(t) for t in (x, w, r, dy, pre, u))
    lay = Z.ZERO_W_KN if kn else Z.ZERO_W_NK
    for out in (BF, F32):
        Y, PRE = mk(torch.zeros(m, n, dtype=out)), mk(torch.zeros(m, n, dtype=BF))
        ep = Z.linear_epilogue(act=Z.ZERO_ACT_SILU, pre=PRE.t, ldpre=PRE.ld, residual=Q.t, ldres=Q.ld)
        Z.zero_linear(X.t, X.ld, W.t, W.ld, lay, m, n, k, ep, Y.t, Y.ld, code(Z, out))
        y, z, ey, ez = R.linear(x, w, kn, None, "silu", residual=r)
        R.assert_within(Y.t, y, ey, "y")
        R.assert_within(PRE.t, z, ez, "pre")
        DX, DU = mk(torch.zeros(m, k, dtype=out)), mk(torch.zeros(m, k, dtype=BF))
        ag = Z.linear_act_grad(Z.ZERO_ACT_GELU, P.t, P.ld, U.t, U.ld, DU.t, DU.ld)
        Z.zero_linear_dinput(DY.t, DY.ld, W.t, W.ld, lay, m, n, k, ag, DX.t, DX.ld, code(Z, out))
        dx, du, ex, eu = R.linear_dinput(dy, w, kn, "gelu", pre, u)
        R.assert_within(DX.t, dx, ex, "dx")
        R.assert_within(DU.t, du, eu, "dgate")
        DW, DB = mk(torch.zeros(w.shape, dtype=out)), mk(torch.zeros(1, n, dtype=out))
        Z.zero_linear_dweight(DY.t, DY.ld, X.t, X.ld, m, n, k, lay, DW.t, DW.ld, code(Z, out),
                              DB.t[0], code(Z, out), False)
        dw, db, ew, eb = R.linear_dweight(dy, x, kn)
        R.assert_within(DW.t, dw, ew, "dw")
        R.assert_within(DB.t[0], db, eb, "dbias")
        for what, t in (("y", Y), ("pre", PRE), ("dx", DX), ("dgate", DU), ("dw", DW), ("dbias", DB)):
            t.check(what)


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("m,n,k,pad", [(2100, 2500, 72, 0), (2100, 2500, 840, 4), (2050, 2563, 90, 0)])
def test_more_tiles_than_the_gpu_holds(cuda, Z, m, n, k, pad, kn):
    """Several tiles per pair of CTAs, the last ragged both ways: sums in turn,
    boxes and masks carried over, fp32 rounds, bias tiles of their own."""
    run_linear(Z, m, n, k, kn, bias=BF, act="gelu_tanh", pre=True, gate=True, p=0.1, residual=BF, pad=pad)
    run_linear(Z, m, n, k, kn, bias=F32, act="silu", residual=F32, out=F32, pad=pad)
    check_dinput(Z, m, k, n, kn, "silu", True, BF, pad, 0)
    check_dinput(Z, m, k, n, kn, "gelu", False, F32, pad, 0)
    check_dweight(Z, k, n, m, kn, BF, BF, True, pad, 0)
    check_dweight(Z, k, n, m, kn, F32, F32, False, pad, 0)


def test_chain_of_products(cuda, Z):
    """Each product reads what the one before wrote and starts before it ends;
    none is waited for on the host."""
    g = torch.Generator(device="cuda").manual_seed(3)
    for m, n in ((1500, 1800), (200, 512), (3, 1024)):
        a = torch.randn(m, n, device="cuda", generator=g).to(BF)
        w = (torch.randn(n, n, device="cuda", generator=g) * n ** -0.5).to(BF)
        outs = [torch.zeros(m, n, dtype=BF, device="cuda") for _ in range(6)]
        src = a
        for y in outs:
            Z.zero_linear(src, n, w, n, Z.ZERO_W_NK, m, n, n, None, y, n)
            src = y
        src = a
        for y in outs:
            want = src.double() @ w.double().T
            assert ((y.double() - want).norm() / want.norm()).item() < R.U16
            src = y


@pytest.mark.parametrize("p", [0.0, 1.0, 0.9999])
def test_linear_dropout_extremes(cuda, Z, p):
    run_linear(Z, 65, 70, 80, True, p=p, residual=BF)


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
def test_linear_without_inputs(cuda, Z, kn):
    """k = 0: y is the epilogue of the bias alone; m or n = 0: nothing."""
    run_linear(Z, 9, 40, 0, kn, bias=BF, act="silu")
    run_linear(Z, 200, 300, 0, kn)
    for m, n in ((0, 8), (8, 0)):
        Y = Guarded(max(m, 1), max(n, 1), BF)
        x = torch.zeros(8, 8, dtype=BF, device="cuda")
        Z.zero_linear(x, 8, x, 8, Z.ZERO_W_KN if kn else Z.ZERO_W_NK, m, n, 8, None, Y.t, 8)
        torch.cuda.synchronize()
        assert bool((Y.buf == -77.0).all())


@pytest.mark.parametrize("m,n,k", [(16, 96, 9000), (300, 264, 9000), (300, 259, 9001), (700, 2048, 8192)])
def test_fp32_results_of_long_sums(cuda, Z, m, n, k):
    """The tensor cores' additions truncate: each of the 48 of a round of 768
    terms loses half a unit in the last place (2^-24 of the running sum) on
    average, and rounds are added to nearest.  So the error of an fp32 result,
    in 2-norms, stays below 48 * 2^-24 = 2.9e-6 however long the sum."""
    g = torch.Generator().manual_seed(6)
    x, w, dy = (randn(g, *s).cuda() for s in ((m, k), (n, k), (k, n)))
    y, dw, db = torch.empty(m, n, device="cuda"), torch.empty(n, m, device="cuda"), torch.empty(n, device="cuda")
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()  # noqa: E731
    Z.zero_linear(x, k, w, k, 0, m, n, k, None, y, n, Z.ZERO_F32)
    assert rel(y, x.double() @ w.double().T) < 2.9e-6
    Z.zero_linear_dinput(x, k, w.T.contiguous(), n, 0, m, k, n, None, y, n, Z.ZERO_F32)
    assert rel(y, x.double() @ w.double().T) < 2.9e-6
    xt = x.T.contiguous()
    for kn in (0, 1):
        out = dw if not kn else dw.view(m, n)
        Z.zero_linear_dweight(dy, n, xt, m, k, n, m, kn, out, n if kn else m, Z.ZERO_F32, db,
                              Z.ZERO_F32)
        want = xt.double().T @ dy.double()
        assert rel(out, want if kn else want.T) < 2.9e-6
        assert rel(db, dy.double().sum(0)) < 2.9e-6


def test_linear_dropped_elements_hide_infinities(cuda, Z):
    """A dropped element contributes exactly 0, whatever the product holds;
    NaN and infinities reach the kept ones, in their own rows alone."""
    m, n, k = 64, 64, 64
    x = torch.zeros(m, k, dtype=BF, device="cuda")
    x[3, 5], x[7, 1] = float("inf"), float("nan")
    w = torch.ones(n, k, dtype=BF, device="cuda")
    y = torch.empty(m, n, dtype=F32, device="cuda")
    ep = Z.linear_epilogue(dropout=Z.dropout_rng(0.5, 5, 6))
    Z.zero_linear(x, k, w, k, Z.ZERO_W_NK, m, n, k, ep, y, n, Z.ZERO_F32)
    keep = R.keep_mask(m, n, 0.5, 5, 6)
    y = cpu(y)
    assert (y[~keep] == 0).all()
    assert torch.isinf(y[3][keep[3]]).all() and torch.isnan(y[7][keep[7]]).all()
    rest = [i for i in range(m) if i not in (3, 7)]
    assert (y[rest] == 0).all()


def test_linear_same_bits_every_time_and_on_any_stream(cuda, Z):
    g = torch.Generator().manual_seed(11)
    m, n, k = 96, 512, 4096
    x, w = randn(g, m, k).cuda(), randn(g, n, k, scale=0.02).cuda()
    a, b = (torch.empty(m, n, dtype=F32, device="cuda") for _ in range(2))
    Z.zero_linear(x, k, w, k, 0, m, n, k, None, a, n, Z.ZERO_F32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(s):
            b.fill_(-1)
            Z.zero_linear(x, k, w, k, 0, m, n, k, None, b, n, Z.ZERO_F32)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(a, b)


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_dinput(cuda, Z, m, n, k, kn):
    for act, gate, out, pad, skew in ((None, False, BF, 0, 0), (None, False, F32, 0, 0),
                                      ("gelu_tanh", False, BF, 0, 0), ("silu", True, BF, 8, 0),
                                      ("relu", True, F32, 1, 1)):
        check_dinput(Z, m, n, k, kn, act, gate, out, pad, skew)


def check_dinput(Z, m, n, k, kn, act, gate, out, pad, skew):
    g = torch.Generator().manual_seed(m + 3 * n + 5 * k)
    mk = lambda t: Guarded(t.shape[0], t.shape[1], t.dtype, pad, skew, t)  # noqa: E731
    dy, w = randn(g, m, n), randn(g, *((k, n) if kn else (n, k)), scale=1 / math.sqrt(n))
    pre, u = randn(g, m, k), randn(g, m, k)
    DY, W, P, U = mk(dy), mk(w), mk(pre), mk(u)
    DX, DU = Guarded(m, k, out, pad, skew), Guarded(m, k, BF, pad, skew)
    ag = None
    if act is not None:
        ag = Z.linear_act_grad(acts(Z)[act], P.t, P.ld, U.t if gate else None, U.ld if gate else 0,
                               DU.t if gate else None, DU.ld if gate else 0)
    Z.zero_linear_dinput(DY.t, DY.ld, W.t, W.ld, Z.ZERO_W_KN if kn else Z.ZERO_W_NK, m, n, k, ag,
                         DX.t, DX.ld, code(Z, out))
    torch.cuda.synchronize()
    dx, du, ex, eu = R.linear_dinput(dy, w, kn, act, pre, u if gate else None)
    R.assert_within(DX.t, dx, ex, "dx")
    DX.check("dx")
    if gate:
        R.assert_within(DU.t, du, eu, "dgate")
    DU.check("dgate")


@pytest.mark.parametrize("act", R.ACTS)
def test_linear_dinput_activations(cuda, Z, act):
    check_dinput(Z, 140, 96, 200, False, act, False, F32, 0, 0)
    check_dinput(Z, 140, 96, 200, True, act, True, BF, 0, 0)


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("m,n,k", SIZES + [(3000, 192, 256), (4100, 40, 24)])
def test_linear_dweight(cuda, Z, m, n, k, kn):
    for out, bias, acc, pad, skew in ((BF, BF, False, 0, 0), (F32, F32, True, 0, 0),
                                      (BF, None, True, 8, 0), (F32, BF, False, 1, 1)):
        check_dweight(Z, m, n, k, kn, out, bias, acc, pad, skew)


def check_dweight(Z, m, n, k, kn, out, bias, acc, pad, skew):
    g = torch.Generator().manual_seed(m + 3 * n + 5 * k)
    mk = lambda t: Guarded(t.shape[0], t.shape[1], t.dtype, pad, skew, t)  # noqa: E731
    dy, x = randn(g, m, n), randn(g, m, k)
    dw0 = randn(g, *((k, n) if kn else (n, k)), dtype=out)
    DY, X = mk(dy), mk(x)
    DW = mk(dw0) if acc else Guarded(*dw0.shape, out, pad, skew)
    db0 = None if bias is None else randn(g, 1, n, dtype=bias)
    DB = None if bias is None else Guarded(1, n, bias, 0, skew, db0 if acc else None)
    Z.zero_linear_dweight(DY.t, DY.ld, X.t, X.ld, m, n, k, Z.ZERO_W_KN if kn else Z.ZERO_W_NK,
                          DW.t, DW.ld, code(Z, out), None if DB is None else DB.t[0],
                          code(Z, bias), acc)
    torch.cuda.synchronize()
    dw, db, ew, eb = R.linear_dweight(dy, x, kn, dw0 if acc else None,
                                      db0[0] if acc and bias is not None else None)
    R.assert_within(DW.t, dw, ew, "dw")
    DW.check("dw")
    if DB is not None:
        R.assert_within(DB.t[0], db, eb, "dbias")
        DB.check("dbias")


def test_linear_dweight_of_no_rows(cuda, Z):
    """m = 0: the gradients are 0, or stay as they were when accumulated to."""
    for acc in (False, True):
        dw = torch.full((24, 40), 3.0, dtype=BF, device="cuda")
        db = torch.full((24,), 5.0, dtype=F32, device="cuda")
        Z.zero_linear_dweight(None, 24, None, 40, 0, 24, 40, 0, dw, 40, Z.ZERO_BF16, db, Z.ZERO_F32,
                              acc)
        assert bool((dw == (3.0 if acc else 0.0)).all()) and bool((db == (5.0 if acc else 0.0)).all())


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
def test_linear_dweight_of_no_inputs(cuda, Z, kn):
    """k = 0: there is no weight, but the bias still has its gradient."""
    m, n = 70, 300
    dy = randn(torch.Generator().manual_seed(5), m, n)
    db = torch.zeros(n, device="cuda")
    Z.zero_linear_dweight(dy.cuda(), n, None, 0, m, n, 0, Z.ZERO_W_KN if kn else Z.ZERO_W_NK, None,
                          n if kn else 0, Z.ZERO_BF16, db, Z.ZERO_F32)
    _, want, _, err = R.linear_dweight(dy, torch.zeros(m, 0), kn)
    R.assert_within(db, want, err, "dbias")


def test_gradients_against_differences(cuda, Z):
    """The kernels' gradients along random directions against central
    differences of the 64-bit forward formulas (values, not slopes, of the
    activation): a gated product after a SiLU."""
    g = torch.Generator().manual_seed(21)
    m, n, k = 48, 72, 80
    z, u, w, c = randn(g, m, k), randn(g, m, k), randn(g, k, n, scale=0.1), randn(g, m, n)
    D = R.D
    x = (R.act(z.to(D), "silu")[0] * u.to(D)).to(BF)

    def loss(z, u, w):
        return (c.to(D) * (R.act(z, "silu")[0] * u @ w)).sum()

    dev = [t.cuda() for t in (z, u, w, c, x)]
    dx, du = torch.empty(m, k, dtype=F32, device="cuda"), torch.empty(m, k, dtype=BF, device="cuda")
    ag = Z.linear_act_grad(Z.ZERO_ACT_SILU, dev[0], k, dev[1], k, du, k)
    Z.zero_linear_dinput(dev[3], n, dev[2], n, Z.ZERO_W_KN, m, n, k, ag, dx, k, Z.ZERO_F32)
    dw = torch.empty(k, n, dtype=F32, device="cuda")
    Z.zero_linear_dweight(dev[3], n, dev[4], k, m, n, k, Z.ZERO_W_KN, dw, n, Z.ZERO_F32)
    args = [t.to(D) for t in (z, u, w)]
    for grad, i, u_round in ((dx, 0, 1e-5), (du, 1, R.U16), (dw, 2, R.U16)):  # dw: of x rounded to bf16
        d = torch.randn(args[i].shape, generator=g, dtype=D)
        h = 1e-5
        up, dn = (loss(*[a + s * h * d if j == i else a for j, a in enumerate(args)]) for s in (1, -1))
        want = (up - dn) / (2 * h)
        gc = cpu(grad).to(D)
        got = (gc * d).sum()
        # each element is off by at most its rounding, and independently: 6 standard deviations
        assert abs(got - want) <= 6 * u_round * (gc * d).norm() + 1e-6 * abs(want)


# ----------------------------------------------------------------- dropout --
@pytest.mark.parametrize("m,n", [(1, 1), (1, 8), (3, 7), (5, 64), (17, 129), (64, 1024), (257, 771),
                                 (1000, 12), (2, 20011)])
@pytest.mark.parametrize("pad,skew", [(0, 0), (1, 0), (8, 8), (0, 3)])
def test_dropout(cuda, Z, m, n, pad, skew):
    g = torch.Generator().manual_seed(m * 5 + n)
    for xt, rt, yt, p in ((BF, BF, BF, 0.1), (F32, None, F32, 0.5), (BF, F32, F32, 0.9),
                          (F32, BF, BF, 0.0), (BF, BF, BF, 1.0)):
        x = randn(g, m, n, dtype=xt)
        r = None if rt is None else randn(g, m, n, dtype=rt)
        X, Y = Guarded(m, n, xt, pad, skew, x), Guarded(m, n, yt, pad, skew)
        Rs = None if rt is None else Guarded(m, n, rt, pad, skew, r)
        seed, off = 2 ** 63 + 12345, 2 ** 40 + 7
        Z.zero_dropout(X.t, X.ld, code(Z, xt), Rs.t if Rs else None, Rs.ld if Rs else 0,
                       code(Z, rt), m, n, Z.dropout_rng(p, seed, off), Y.t, Y.ld, code(Z, yt))
        want = R.drop(x.to(R.D), p, seed, off)
        err = 4 * R.U32 * want.abs()
        if r is not None:
            want = want + r.to(R.D)
            err = err + R.U32 * want.abs()
        R.assert_within(Y.t, want, err, "y")
        Y.check("y")


def test_dropout_in_place_and_offsets(cuda, Z):
    """y may be x or the residual; a device offset adds to the host's, and a
    replayed graph draws a new mask when it changes; the product's epilogue
    draws the mask this call draws."""
    g = torch.Generator().manual_seed(2)
    m, n = 40, 100
    x, r = randn(g, m, n, dtype=F32), randn(g, m, n, dtype=F32)
    for alias in ("x", "r"):
        X, Q = x.cuda(), r.cuda()
        y = X if alias == "x" else Q
        Z.zero_dropout(X, n, 0, Q, n, 0, m, n, Z.dropout_rng(0.3, 4, 5), y, n, 0)
        want = R.drop(x.to(R.D), 0.3, 4, 5) + r.to(R.D)
        R.assert_within(y, want, 6 * R.U32 * (want.abs() + r.to(R.D).abs()), alias)
    d_off = torch.tensor([2 ** 33], dtype=torch.int64, device="cuda")
    X, y = x.cuda(), torch.empty(m, n, device="cuda")
    rng = Z.dropout_rng(0.3, 4, 5, d_off)
    Z.zero_dropout(X, n, 0, None, 0, 0, m, n, rng, y, n, 0)       # warm up
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        Z.zero_dropout(X, n, 0, None, 0, 0, m, n, rng, y, n, 0)
    for off in (1, 2 ** 33, -1):
        d_off.fill_(off)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cpu(y) != 0, R.keep_mask(m, n, 0.3, 4, 5 + off))
    k = 16
    a, w = torch.ones(m, k, dtype=BF, device="cuda"), torch.ones(n, k, dtype=BF, device="cuda")
    ep = Z.linear_epilogue(dropout=Z.dropout_rng(0.3, 4, 7))
    Z.zero_linear(a, k, w, k, 0, m, n, k, ep, y, n, Z.ZERO_F32)
    assert torch.equal(cpu(y) != 0, R.keep_mask(m, n, 0.3, 4, 7))


def test_dropout_hides_nan_and_infinity(cuda, Z):
    m, n = 33, 65
    x = torch.full((m, n), float("nan"), device="cuda")
    x[::2] = float("inf")
    y = torch.empty(m, n, device="cuda")
    Z.zero_dropout(x, n, 0, None, 0, 0, m, n, Z.dropout_rng(0.5, 1, 2), y, n, 0)
    keep = R.keep_mask(m, n, 0.5, 1, 2)
    y = cpu(y)
    assert (y[~keep] == 0).all() and not torch.isfinite(y[keep]).any()


# -------------------------------------------------------------- layer norm --
NORMS = [(1, 1), (1, 8), (3, 33), (9, 256), (7, 257), (20, 512), (11, 771), (33, 1024), (5, 1025),
         (130, 2048), (6, 4096), (3, 5504), (700, 96), (2, 8200), (3, 16384), (2, 16385), (40, 20000)]


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("m,n", NORMS)
def test_layer_norm(cuda, Z, m, n, rms):
    g = torch.Generator().manual_seed(m + n)
    kind = Z.ZERO_NORM_RMS if rms else Z.ZERO_NORM_LAYER
    for xt, pt, yt, has_b, pad, skew in ((BF, BF, BF, True, 0, 0), (F32, F32, F32, False, 0, 0),
                                         (BF, F32, F32, True, 1, 3), (F32, BF, BF, True, 8, 8)):
        x = (randn(g, m, n, dtype=F32) + 3.0).to(xt)
        w, b = randn(g, n, dtype=pt), randn(g, n, dtype=pt) if has_b else None
        X, Y = Guarded(m, n, xt, pad, skew, x), Guarded(m, n, yt, pad, skew)
        W = Guarded(1, n, pt, 0, skew, w[None])
        Bv = None if b is None else Guarded(1, n, pt, 0, skew, b[None])
        mean = None if rms else torch.full((m,), -7.0, device="cuda")
        rstd = torch.full((m,), -7.0, device="cuda")
        Z.zero_layer_norm(X.t, X.ld, code(Z, xt), W.t[0], Bv.t[0] if Bv else None, code(Z, pt), m, n,
                          kind, 1e-5, Y.t, Y.ld, code(Z, yt), mean, rstd)
        y, mu, rs, ey = R.norm(x, w, b, rms, 1e-5)
        R.assert_within(Y.t, y, ey, "y")
        Y.check("y")
        if n > 1:                      # with one element layer norm's rstd is 1/sqrt(eps) exactly
            depth = 40 + n / 256
            R.assert_within(rstd, rs, depth * R.U32 * rs * (1 + x.to(R.D).abs().mean(1) * rs), "rstd")
        if mean is not None:
            R.assert_within(mean, mu, (24 + n / 256) * R.U32 * x.to(R.D).abs().mean(1), "mean")


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("m,n", [s for s in NORMS if s[1] > 1] + [(2500, 128), (1300, 1032)])
def test_layer_norm_backward(cuda, Z, m, n, rms):
    g = torch.Generator().manual_seed(m + n)
    kind = Z.ZERO_NORM_RMS if rms else Z.ZERO_NORM_LAYER
    for xt, pt, has_b, res, acc, pad, skew in ((BF, BF, True, True, False, 0, 0),
                                               (F32, F32, False, False, True, 0, 0),
                                               (BF, F32, True, True, True, 1, 3),
                                               (F32, BF, True, False, False, 8, 8)):
        x, dy = (randn(g, m, n, dtype=F32) + 1.0).to(xt), randn(g, m, n, dtype=xt)
        w, r = randn(g, n, dtype=pt), randn(g, m, n, dtype=xt) if res else None
        dw0, db0 = randn(g, n, dtype=pt), randn(g, n, dtype=pt)
        _, mu, rs, _ = R.norm(x, w, None, rms, 1e-5)
        mean, rstd = (None if rms else mu.float().cuda()), rs.float().cuda()
        X, DY, W = (Guarded(t.shape[0], n, t.dtype, pad if t.shape[0] > 1 else 0, skew, t)
                    for t in (x, dy, w[None]))
        DX = Guarded(m, n, xt, pad, skew, r)                 # dres in place
        DW = Guarded(1, n, pt, 0, skew, dw0[None] if acc else None)
        DB = Guarded(1, n, pt, 0, skew, db0[None] if acc else None) if has_b else None
        size = Z.zero_layer_norm_workspace(m, n)
        ws = torch.full((size // 4 + 8,), float("nan"), device="cuda")
        Z.zero_layer_norm_backward(DY.t, DY.ld, code(Z, xt), X.t, X.ld, code(Z, xt), W.t[0],
                                   code(Z, pt), mean, rstd, m, n, kind, DX.t if res else None,
                                   DX.ld if res else 0, DX.t, DX.ld, code(Z, xt), DW.t[0],
                                   DB.t[0] if DB else None, code(Z, pt), acc, ws, size)
        dx, dw, db, ex, ew, eb = R.norm_backward(
            dy, x, w, None if rms else cpu(mean), cpu(rstd), rms, r, dw0 if acc else None,
            db0 if acc else None)
        R.assert_within(DX.t, dx, ex, "dx")
        R.assert_within(DW.t[0], dw, ew, "dweight")
        if DB:
            R.assert_within(DB.t[0], db, eb, "dbias")
            DB.check("dbias")
        DX.check("dx")
        DW.check("dweight")
        assert bool(torch.isnan(ws[size // 4:]).all()), "wrote past the workspace"


def test_layer_norm_of_constant_rows_and_none(cuda, Z):
    """A row of equal values normalises to the bias; no rows: gradients 0."""
    m, n = 5, 1000
    x = torch.full((m, n), 1e4, device="cuda")
    w, b = torch.ones(n, device="cuda"), torch.full((n,), 0.5, device="cuda")
    y, rstd = torch.empty(m, n, device="cuda"), torch.empty(m, device="cuda")
    Z.zero_layer_norm(x, n, 0, w, b, 0, m, n, 0, 1e-5, y, n, 0, None, rstd)
    # the mean of 1000 equal values is off by a few ulps of 1e4, which rstd <= 316 magnifies
    assert (y - 0.5).abs().max().item() <= 16 * R.U32 * 1e4 * 317
    dw, db = torch.full((n,), 3.0, device="cuda"), torch.full((n,), 4.0, device="cuda")
    Z.zero_layer_norm_backward(None, n, 0, None, n, 0, w, 0, None, None, 0, n, 0, None, 0, None, n,
                               0, dw, db, 0, False, None, 0)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_layer_norm_in_place_same_bits(cuda, Z):
    g = torch.Generator().manual_seed(8)
    for m, n in ((50, 768), (9, 4096), (3, 20000)):
        x, w = randn(g, m, n).cuda(), randn(g, n).cuda()
        y = torch.empty_like(x)
        Z.zero_layer_norm(x, n, 1, w, w, 1, m, n, 0, 1e-5, y, n, 1)
        Z.zero_layer_norm(x, n, 1, w, w, 1, m, n, 0, 1e-5, x, n, 1)
        assert torch.equal(x, y)
