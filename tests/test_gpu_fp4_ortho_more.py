"""4-bit layers and orthogonalised updates as a program uses them: a training
step of both on a plan's flat buffers, eager and replayed from a graph; few rows
against many; calls at once; places beyond 32 bits."""
import math

import pytest
import torch

import fp4_reference as Q
import ops_reference as R
import ortho_reference as O
from test_gpu_fp4 import Packed, fmt, operand, run_linear
from test_gpu_ops import randn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_optimizer_device_gb300 as Z
    return Z


# ------------------------------------------------------------ a training step --
class Layer:
    """y = gelu_tanh(x W1^T) W2^T in 4 bits, trained on the gradients of two
    ranks (each half of the rows): quantise, forward, backward, reduce-scatter,
    step.  Every stage's inputs stay in reach of the test."""

    def __init__(self, Z, form, m, d, h):
        self.Z, self.form, self.f, self.m, self.d, self.h = Z, form, fmt(Z, form), m, d, h
        self.plan = Z.zero_plan([8, h * d, 16, d * h], 2, 16)
        self.P = Z.zero_plan_info(self.plan)["psi_pad"]
        self.at = [Z.zero_plan_tensor(self.plan, t)[0] for t in (1, 3)]
        g = torch.Generator().manual_seed(17)
        dev = lambda t: t.cuda()  # noqa: E731
        self.master = dev(torch.randn(self.P, generator=g) * 0.05)
        self.momentum = dev(torch.zeros(self.P))
        self.reduced = dev(torch.zeros(self.P))
        self.params = self.master.to(BF)
        self.x, self.target = dev(randn(g, m, d)), dev(randn(g, m, d))
        new = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")  # noqa: E731
        self.z, self.a, self.y, self.dy, self.dz = new(m, h), new(m, h), new(m, d), new(m, d), new(m, h)
        self.grads = [new(self.P) for _ in range(2)]
        self.work = torch.empty(Z.ZERO_FP4_WORKSPACE, dtype=torch.uint8, device="cuda")
        self.room = {}
        self.sizes = {(h, d): Z.zero_muon_workspace(h, d, 1), (d, h): Z.zero_muon_workspace(d, h, 1)}
        self.scratch = torch.empty(max(self.sizes.values()), dtype=torch.uint8, device="cuda")
        self.hp = Z.muon_hp(lr=0.02, weight_decay=0.1, grad_scale=0.5)

    def quant(self, name, x, rows, cols, both):
        """x's 4-bit forms: along its rows, and along its columns."""
        Z = self.Z
        if name not in self.room:
            g = torch.zeros(1, device="cuda") if self.form == "nv" else None
            self.room[name] = (Packed(Z, rows, cols, self.form, 0, g), Packed(Z, cols, rows, self.form, 0, g), g)
        q, qt, g = self.room[name]
        if g is not None:
            Z.zero_fp4_tensor_scale(x, cols, Z.ZERO_BF16, rows, cols, g, self.work, self.work.numel())
        Z.zero_fp4_quantize(x, cols, Z.ZERO_BF16, rows, cols, self.f, q.mat if both != "t" else None, qt.mat if both else None)
        return q.mat, qt.mat

    def weight(self, i, flat):
        rows, cols = ((self.h, self.d), (self.d, self.h))[i]
        return flat[self.at[i]:self.at[i] + rows * cols].view(rows, cols)

    def step(self):
        Z, f, m, d, h = self.Z, self.f, self.m, self.d, self.h
        w1, w1t = self.quant("w1", self.weight(0, self.params), h, d, True)
        w2, w2t = self.quant("w2", self.weight(1, self.params), d, h, True)
        x, _ = self.quant("x", self.x, m, d, False)
        Z.zero_fp4_linear(x, w1, f, m, h, d, Z.linear_epilogue(act=Z.ZERO_ACT_GELU_TANH, pre=self.z, ldpre=h), self.a, h)
        a, _ = self.quant("a", self.a, m, h, False)
        Z.zero_fp4_linear(a, w2, f, m, d, h, None, self.y, d)
        torch.sub(self.y, self.target, out=self.dy)
        dy, _ = self.quant("dy", self.dy, m, d, False)
        Z.zero_fp4_linear_dinput(dy, w2t, f, m, d, h, Z.linear_act_grad(Z.ZERO_ACT_GELU_TANH, self.z, h), self.dz, h)
        half = m // 2
        for r in range(2):
            part = slice(r * half, (r + 1) * half)
            _, dyt = self.quant(f"dyt{r}", self.dy[part], half, d, "t")
            _, at = self.quant(f"at{r}", self.a[part], half, h, "t")
            Z.zero_fp4_linear_dweight(dyt, at, f, half, d, h, self.weight(1, self.grads[r]), h)
            _, dzt = self.quant(f"dzt{r}", self.dz[part], half, h, "t")
            _, xt = self.quant(f"xt{r}", self.x[part], half, d, "t")
            Z.zero_fp4_linear_dweight(dzt, xt, f, half, h, d, self.weight(0, self.grads[r]), d)
        Z.zero_reduce_scatter(self.plan, 0, self.grads, Z.ZERO_BF16, self.reduced, 0, self.P, 1.0)
        for t, rows, cols in ((1, h, d), (3, d, h)):
            Z.zero_muon_step(self.plan, [t], rows, cols, self.master, self.momentum, self.reduced, self.hp, None, self.params, Z.ZERO_BF16, self.scratch,
                             self.sizes[rows, cols])

    def values(self, x):
        """What x stands for once quantised along its rows, in 64 bits."""
        x = x.cpu().float()
        return Q.quantise(x, self.form, Q.tensor_scale(x) if self.form == "nv" else None)[2]


@pytest.mark.parametrize("form", ["mx", "nv"])
def test_training_step(cuda, Z, form):
    L = Layer(Z, form, 96, 72, 136)
    L.step()                                               # momentum and other weights than the first
    before = [t.clone() for t in (L.params, L.master, L.momentum)]
    L.step()
    torch.cuda.synchronize()
    w1, w2 = (L.weight(i, before[0]) for i in (0, 1))
    y, z, ey, ez = R.linear(L.values(L.x), L.values(w1), False, None, "gelu_tanh")
    R.assert_within(L.a, y, ey, "a")
    R.assert_within(L.z, z, ez, "z")
    y, _, ey, _ = R.linear(L.values(L.a), L.values(w2), False)
    R.assert_within(L.y, y, ey, "y")
    dz, _, e, _ = R.linear_dinput(L.values(L.dy), L.values(w2.t()), True, "gelu_tanh", L.z.cpu())
    R.assert_within(L.dz, dz, e, "dz")
    for r in range(2):
        p = slice(r * 48, (r + 1) * 48)
        for i, (out, inp) in enumerate(((L.dz, L.x), (L.dy, L.a))):
            dw, _, e, _ = R.linear_dweight(L.values(out[p].t()).T, L.values(inp[p].t()).T, False)
            R.assert_within(L.weight(i, L.grads[r]), dw, e, f"dw{i + 1} of rank {r}")
    f = lambda v: torch.tensor(v, dtype=F32)  # noqa: E731
    for i in (0, 1):
        ring = L.weight(i, L.grads[0]).cpu().float() + L.weight(i, L.grads[1]).cpu().float()
        assert torch.equal(L.weight(i, L.reduced).cpu(), ring)
        grad = ring * f(0.5)
        mom = f(0.95) * L.weight(i, before[2]).cpu() + grad
        assert torch.equal(L.weight(i, L.momentum).cpu(), mom)
        o, off = O.allowance(grad + f(0.95) * mom)
        lr, wd, old = f(0.02).double(), f(0.1).double(), L.weight(i, before[1]).cpu().double()
        want = old * (1 - lr * wd) - lr * o
        got = L.weight(i, L.master).cpu()
        assert (got.double() - want).norm() <= lr * (off + 2.0 ** -11 * o.norm()) + 3 * 2.0 ** -24 * old.norm()
        assert torch.equal(L.weight(i, L.params).cpu(), got.to(BF))


def test_training_step_from_a_graph(cuda, Z):
    """Captured and replayed, the step leaves the bits that eager steps leave."""
    a, b = (Layer(Z, "nv", 64, 40, 72) for _ in range(2))
    for _ in range(4):
        a.step()
    b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for x, y in ((a.master, b.master), (a.momentum, b.momentum), (a.params, b.params), (a.y, b.y)):
        assert torch.equal(x, y)


# ------------------------------------------------------------------- few rows --
@pytest.mark.parametrize("form", ["mx", "nv"])
@pytest.mark.parametrize("n,k", [(1, 4099), (31, 32), (33, 40), (127, 1000), (129, 64), (260, 2056), (520, 9000), (2000, 700)])
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 7, 8, 9])
def test_few_rows(cuda, Z, m, n, k, form):
    """Every count of rows, outputs that end inside a group of four and a tile
    of 128, contractions of a piece of a warp's and of many."""
    run_linear(Z, m, n, k, form, bias=F32, act="silu", pre=True, gate=True, residual=BF, p=0.25)
    run_linear(Z, m, n, k, form, out=F32, pad=1, skew=3)


@pytest.mark.parametrize("form", ["mx", "nv"])
def test_few_rows_and_many_agree(cuda, Z, form):
    """A row's result does not depend on how many come with it, up to fp32 sums:
    both within 2 (k + 4) units of the sum of magnitudes."""
    g = torch.Generator().manual_seed(23)
    m, n, k = 40, 300, 1000
    x, vx, gx = operand(Z, g, m, k, form)
    w, vw, gw = operand(Z, g, n, k, form)
    many, few = torch.empty(m, n, device="cuda"), torch.empty(8, n, device="cuda")
    Z.zero_fp4_linear(x.mat, w.mat, fmt(Z, form), m, n, k, None, many, n, Z.ZERO_F32)
    Z.zero_fp4_linear(x.mat, w.mat, fmt(Z, form), 8, n, k, None, few, n, Z.ZERO_F32)
    size = (vx[:8].abs() @ vw.T.abs()) * (gx * gw)
    assert ((many[:8] - few).abs().cpu().double() <= 2 * (k + 4) * R.U32 * size).all()


@pytest.mark.parametrize("m", [1, 5, 100])
def test_nan_scales_in_a_weight(cuda, Z, m):
    g = torch.Generator().manual_seed(29)
    for form, bad in (("mx", 255), ("nv", 127)):
        n, k = 200, 300
        x, _, _ = operand(Z, g, m, k, form)
        w = torch.randn(n, k, generator=g)
        c, b, _ = Q.quantise(w, form)
        b[7, 1], b[199, -1] = bad, bad
        W = Packed(Z, n, k, form, 0, None if form == "mx" else torch.ones(1, device="cuda")).fill(c, b)
        y = torch.empty(m, n, device="cuda")
        Z.zero_fp4_linear(x.mat, W.mat, fmt(Z, form), m, n, k, None, y, n, Z.ZERO_F32)
        want = torch.zeros(m, n, dtype=torch.bool)
        want[:, 7] = want[:, 199] = True
        assert torch.equal(torch.isnan(y).cpu(), want)


@pytest.mark.parametrize("m", [1, 6, 200])
def test_scales_at_both_ends(cuda, Z, m):
    """Block scales of 2^-100 against 2^100: their product is exact, whatever either alone does to a partial product; zero blocks under a huge scale stay 0."""
    n, k = 130, 128
    g = torch.Generator().manual_seed(31)
    code = lambda r: torch.randint(0, 16, (r, k), generator=g, dtype=torch.uint8)  # noqa: E731
    cx, cw = code(m), code(n)
    bx, bw = torch.full((m, 4), 27, dtype=torch.uint8), torch.full((n, 4), 227, dtype=torch.uint8)
    cx[:, 32:64], bx[:, 1], bw[:, 1] = 0, 254, 254
    x, w = Packed(Z, m, k, "mx").fill(cx, bx), Packed(Z, n, k, "mx").fill(cw, bw)
    y = torch.empty(m, n, device="cuda")
    Z.zero_fp4_linear(x.mat, w.mat, Z.ZERO_FP4_MX, m, n, k, None, y, n, Z.ZERO_F32)
    v = lambda c: Q.LEVELS[(c & 7).long()] * torch.where(c > 7, -1.0, 1.0)  # noqa: E731
    assert torch.equal(y.cpu().double(), v(cx) @ v(cw).T)      # multiples of 1/4 below 2^14: exact in fp32


# -------------------------------------------------- streams, graphs, repeats --
@pytest.mark.parametrize("m", [3, 300])
def test_products_on_two_streams_and_from_a_graph(cuda, Z, m):
    g = torch.Generator().manual_seed(37)
    n, k = 520, 1000
    w, vw, gw = operand(Z, g, n, k, "nv")
    xs = torch.randn(m, k, generator=g).to(BF).cuda()

    def call(scale, q, y, work):
        Z.zero_fp4_tensor_scale(xs, k, Z.ZERO_BF16, m, k, scale, work, work.numel())
        Z.zero_fp4_quantize(xs, k, Z.ZERO_BF16, m, k, Z.ZERO_FP4_NV, q.mat)
        Z.zero_fp4_linear(q.mat, w.mat, Z.ZERO_FP4_NV, m, n, k, None, y, n)

    args = []
    for _ in range(2):
        scale = torch.zeros(1, device="cuda")
        args.append((scale, Packed(Z, m, k, "nv", 0, scale), torch.zeros(m, n, dtype=BF, device="cuda"), torch.empty(4096, dtype=torch.uint8, device="cuda")))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        with torch.cuda.stream(s):
            call(*args[1])
        call(*args[0])
    torch.cuda.synchronize()
    assert torch.equal(args[0][2], args[1][2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*args[1])
    for _ in range(3):
        xs.mul_(-0.75)
        graph.replay()
        call(*args[0])
        torch.cuda.synchronize()
        assert torch.equal(args[0][2], args[1][2])


def test_steps_beside_other_work(cuda, Z):
    """A step waits for nothing but its own tiles while products fill the GPU from another stream."""
    n = 2048
    x = torch.randn(2, 300, 500, device="cuda")
    y, z = (torch.zeros(2, 300, 500, dtype=BF, device="cuda") for _ in range(2))
    size = Z.zero_orthogonalize_workspace(300, 500, 2)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    call = lambda out: Z.zero_orthogonalize(x, 500, 150000, Z.ZERO_F32, 300, 500, 2, Z.newton_schulz(), out, 500, 150000, work, size)  # noqa: E731
    call(y)
    a, c = torch.randn(n, n, device="cuda").to(BF), torch.zeros(n, n, dtype=BF, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(40):
            Z.zero_linear(a, n, a, n, Z.ZERO_W_NK, n, n, n, None, c, n)
    for _ in range(10):
        call(z)
    torch.cuda.synchronize()
    assert torch.equal(y, z)


# ---------------------------------------------------------- beyond 32 bits --
def test_codes_beyond_32_bits(cuda, Z):
    """More than 2^32 values, codes past byte 2^31 in both directions: their last rows and columns against a small matrix's."""
    rows, cols = 40000, 110000
    x = torch.empty(rows, cols, dtype=BF, device="cuda")
    for r in range(0, rows, 4000):
        x[r:r + 4000].normal_(generator=torch.Generator(device="cuda").manual_seed(r))
    row, size = Z.zero_fp4_size(rows, cols, Z.ZERO_FP4_MX)
    row_t, size_t = Z.zero_fp4_size(cols, rows, Z.ZERO_FP4_MX)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    c, s, ct, st = u8(rows, row), u8(size), u8(cols, row_t), u8(size_t)
    assert c.numel() > 2 ** 31 and ct.numel() > 2 ** 31
    q, qt = Z.fp4_matrix(c, row, s), Z.fp4_matrix(ct, row_t, st)
    Z.zero_fp4_quantize(x, cols, Z.ZERO_BF16, rows, cols, Z.ZERO_FP4_MX, q, qt)
    last = x[-64:].clone()                                   # 40000 = 312 * 128 + 64
    small = Packed(Z, 64, cols, "mx")
    Z.zero_fp4_quantize(last, cols, Z.ZERO_BF16, 64, cols, Z.ZERO_FP4_MX, small.mat)
    assert torch.equal(c[-64:], small.codes) and torch.equal(s[-small.size:], small.scales)
    y = torch.empty(rows, cols, dtype=BF, device="cuda")
    Z.zero_fp4_dequantize(q, rows, cols, Z.ZERO_FP4_MX, y, cols)
    v = torch.empty(64, cols, dtype=BF, device="cuda")
    Z.zero_fp4_dequantize(small.mat, 64, cols, Z.ZERO_FP4_MX, v, cols)
    assert torch.equal(y[-64:], v)
    tail = x[:, -48:].contiguous()                           # 110000 = 859 * 128 + 48
    small = Packed(Z, 48, rows, "mx")
    Z.zero_fp4_quantize(tail, 48, Z.ZERO_BF16, rows, 48, Z.ZERO_FP4_MX, None, small.mat)
    assert torch.equal(ct[-48:], small.codes) and torch.equal(st[-small.size:], small.scales)
    # one row of it against many outputs: the weight's rows lie past 2^31 bytes
    t = Packed(Z, 1, cols, "mx")
    Z.zero_fp4_quantize(last[:1], cols, Z.ZERO_BF16, 1, cols, Z.ZERO_FP4_MX, t.mat)
    for m in (1, 16):
        r = Packed(Z, m, cols, "mx")
        Z.zero_fp4_quantize(last[:m].contiguous(), cols, Z.ZERO_BF16, m, cols, Z.ZERO_FP4_MX, r.mat)
        out = torch.zeros(m, rows, device="cuda")
        Z.zero_fp4_linear(r.mat, q, Z.ZERO_FP4_MX, m, rows, cols, None, out, rows, Z.ZERO_F32)
        want = (v[:m].double() @ v.double().T)
        assert ((out[:, -64:].double() - want).norm() / want.norm()).item() < 2.9e-6


def test_step_on_a_tensor_beyond_32_bits(cuda, Z):
    """A tensor whose elements begin past 2^31 (and its bytes past 2^33)."""
    rows, cols = 60, 72
    numels = [2 ** 31 + 8 * 1000 + 5, rows * cols, 3]
    plan = Z.zero_plan(numels, 8, 16)
    total, at = Z.zero_plan_info(plan)["psi_pad"], Z.zero_plan_tensor(plan, 1)[0]
    master, momentum, reduced = (torch.zeros(total, device="cuda") for _ in range(3))
    out = torch.zeros(total, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(41)
    small = [torch.randn(rows * cols, generator=g) for _ in range(3)]
    s = slice(at, at + rows * cols)
    for big, v in zip((master, momentum, reduced), small):
        big[s] = v.cuda()
    size = Z.zero_muon_workspace(rows, cols, 1)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    hp = Z.muon_hp(lr=0.1)
    Z.zero_muon_step(plan, [1], rows, cols, master, momentum, reduced, hp, None, out, Z.ZERO_BF16, work, size)
    p2 = Z.zero_plan([5, rows * cols], 8, 16)
    n2 = Z.zero_plan_info(p2)["psi_pad"]
    m2, b2, r2 = (torch.zeros(n2, device="cuda") for _ in range(3))
    for big, v in zip((m2, b2, r2), small):
        big[5:5 + rows * cols] = v.cuda()
    Z.zero_muon_step(p2, [1], rows, cols, m2, b2, r2, hp, None, None, Z.ZERO_BF16, work, size)
    for big, v in ((master, m2), (momentum, b2)):
        assert torch.equal(big[s], v[5:5 + rows * cols])
        assert int((big != 0).sum()) <= rows * cols
    assert torch.equal(out[s], m2[5:5 + rows * cols].to(BF)) and int((out != 0).sum()) <= rows * cols


def test_a_matrix_of_many_tiles_down_a_long_side(cuda, Z):
    """50257 x 96, the shape of an embedding: a long contraction into one tile."""
    x = torch.randn(50257, 96, generator=torch.Generator().manual_seed(43)) * 0.01
    y = torch.empty(50257, 96, dtype=BF, device="cuda")
    size = Z.zero_orthogonalize_workspace(50257, 96, 1)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    Z.zero_orthogonalize(x.cuda(), 96, 0, Z.ZERO_F32, 50257, 96, 1, Z.newton_schulz(), y, 96, 0, work, size)
    want, off = O.allowance(x)
    assert (y.cpu().double() - want).norm() <= off + 2.0 ** -8 * want.norm()
    assert math.isfinite(y.float().abs().max().item())
