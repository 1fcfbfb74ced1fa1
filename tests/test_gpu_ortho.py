"""Orthogonalised updates on the GPU against Newton-Schulz steps in 64 bits:
sizes on both sides of the tiles, odd ones, batches, strides, the ends of the
range; the step on the flat arrays element by element."""
import math

import pytest
import torch

import ortho_reference as O
from test_gpu_ops import Guarded, code

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_optimizer_device_gb300 as Z
    return Z


def matrix(g, m, n, kind="random"):
    if kind == "random":
        return torch.randn(m, n, generator=g) * 1e-3
    r = max(1, min(m, n) // 8)           # strong directions over weak ones
    x = torch.randn(m, r, generator=g) * torch.arange(1, r + 1).float().pow(-1.0) @ torch.randn(r, n, generator=g)
    return x + 0.01 * torch.randn(m, n, generator=g)


def scratch(Z, m, n, batch):
    size = Z.zero_orthogonalize_workspace(m, n, batch)
    buf = torch.full((256 + size + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    return buf, buf[256:256 + size], size


def run(Z, xs, dtype=BF, steps=5, coef=O.JORDAN, eps=1e-7, pad=0, skew=0, in_place=False):
    """Orthogonalises a batch and compares each of its matrices."""
    batch, (m, n) = len(xs), xs[0].shape
    rows = torch.cat([x.to(dtype) for x in xs])                  # one below the other, a row between two
    gap = 1 if batch > 1 else 0
    full = torch.zeros(batch * (m + gap), n, dtype=dtype)
    for b in range(batch):
        full[b * (m + gap):b * (m + gap) + m] = rows[b * m:(b + 1) * m]
    X = Guarded(batch * (m + gap), n, dtype, pad, skew, full)
    Y = X if in_place else Guarded(batch * (m + gap), n, BF, pad, skew, torch.full_like(full, 3.0).to(BF))
    stride = (m + gap) * X.ld
    buf, work, size = scratch(Z, m, n, batch)
    Z.zero_orthogonalize(X.t, X.ld, stride, code(Z, dtype), m, n, batch, Z.newton_schulz(steps, coef, eps), Y.t, Y.ld, stride, work, size)
    torch.cuda.synchronize()
    assert bool((buf[:256] == 0x5A).all() and (buf[-256:] == 0x5A).all()), "wrote outside the workspace"
    Y.check("y")
    got = Y.t.cpu().double()
    for b in range(batch):
        want, off = O.allowance(xs[b].to(dtype), steps, coef, eps)
        y = got[b * (m + gap):b * (m + gap) + m]
        bound = off + 2.0 ** -8 * want.norm()
        assert (y - want).norm() <= bound, f"matrix {b}: {(y - want).norm() / want.norm():.3g} off, {bound / want.norm():.3g} allowed"
        if gap:
            left = got[b * (m + gap) + m]
            assert bool((left == (0.0 if in_place else 3.0)).all()), "wrote between two matrices"
    return got


SIZES = [(1, 1), (1, 7), (7, 1), (2, 2), (3, 40), (40, 3), (16, 16), (63, 65), (64, 64), (65, 63), (128, 128), (129, 100), (100, 129), (255, 257), (256, 256),
         (257, 255), (300, 300), (90, 700), (700, 90), (520, 600), (600, 520), (1000, 33), (33, 1000)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,n", SIZES)
def test_one_matrix(cuda, Z, m, n, dtype):
    g = torch.Generator().manual_seed(m * 31 + n)
    run(Z, [matrix(g, m, n)], dtype)
    run(Z, [matrix(g, m, n, "steep")], dtype, pad=1, skew=3)
    run(Z, [matrix(g, m, n)], dtype, pad=8)


@pytest.mark.parametrize("batch,m,n", [(2, 64, 64), (5, 100, 33), (3, 33, 100), (4, 257, 130), (9, 1, 5), (40, 20, 70), (3, 300, 520)])
def test_batches(cuda, Z, batch, m, n):
    g = torch.Generator().manual_seed(batch + m + n)
    for dtype in (BF, F32):
        run(Z, [matrix(g, m, n, ("random", "steep")[b % 2]) * 10.0 ** (b % 5 - 2) for b in range(batch)], dtype, pad=3)
    run(Z, [matrix(g, m, n) for _ in range(batch)], BF, in_place=True)


@pytest.mark.parametrize("m,n", [(1100, 1200), (1200, 1100), (400, 3000), (3000, 400)])
def test_many_tiles(cuda, Z, m, n):
    run(Z, [matrix(torch.Generator().manual_seed(3), m, n, "steep")], F32)


@pytest.mark.parametrize("steps", [0, 1, 2, 6])
def test_steps(cuda, Z, steps):
    x = matrix(torch.Generator().manual_seed(4), 130, 260)
    run(Z, [x], F32, steps)
    run(Z, [x.T.contiguous()], F32, steps)


def test_coefficients_of_each_step(cuda, Z):
    """Degree 3 steps (c = 0) and a sequence of unlike ones."""
    x = matrix(torch.Generator().manual_seed(5), 200, 150)
    run(Z, [x], F32, 6, (1.5, -0.5, 0.0))
    run(Z, [x], F32, 3, [(3.4445, -4.7750, 2.0315), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)])


def test_orthogonal(cuda, Z):
    """With steps that converge, the rows come out orthonormal: G = I to the products' accuracy and y's rounding."""
    x = matrix(torch.Generator().manual_seed(6), 96, 300)
    y = run(Z, [x], F32, 16, (1.875, -1.25, 0.375))
    assert (y @ y.T - torch.eye(96, dtype=torch.float64)).abs().max() < 2 * 2.0 ** -8


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-36, 1e-25, 1e-12, 1e8, 1e20, 1e34])
def test_ends_of_the_range(cuda, Z, size, dtype):
    """Values whose squares leave fp32's range, without eps."""
    x = torch.randn(70, 90, generator=torch.Generator().manual_seed(7)) * size
    run(Z, [x], dtype, eps=0.0)


def test_zeros_nan_and_infinity_keep_to_their_matrix(cuda, Z):
    m, n, batch = 70, 50, 4
    x = torch.randn(batch, m, n, generator=torch.Generator().manual_seed(8))
    x[0] = 0.0
    x[1, 3, 4] = float("nan")
    x[2, 5, 6] = -float("inf")
    for eps in (0.0, 1e-7):
        X, y = x.cuda(), torch.zeros(batch, m, n, dtype=BF, device="cuda")
        _, work, size = scratch(Z, m, n, batch)
        Z.zero_orthogonalize(X, n, m * n, Z.ZERO_F32, m, n, batch, Z.newton_schulz(eps=eps), y, n, m * n, work, size)
        y = y.cpu().double()
        assert bool((y[0] == 0).all() and torch.isnan(y[1]).all() and torch.isnan(y[2]).all())
        want, off = O.allowance(x[3], eps=eps)
        assert (y[3] - want).norm() <= off + 2.0 ** -8 * want.norm()


def test_nothing_to_do(cuda, Z):
    y = torch.full((4, 4), 5.0, dtype=BF, device="cuda")
    x = torch.ones(4, 4, dtype=BF, device="cuda")
    for m, n, batch in ((0, 4, 1), (4, 0, 1), (4, 4, 0)):
        assert Z.zero_orthogonalize_workspace(m, n, batch) == 0
        Z.zero_orthogonalize(x, 4, 16, Z.ZERO_BF16, m, n, batch, Z.newton_schulz(), y, 4, 16, None, 0)
    torch.cuda.synchronize()
    assert bool((y == 5.0).all())


# --------------------------------------------------------------- the step --
def muon_step(Z, numels, tensors, rows, cols, *, nesterov=True, mu=0.95, wd=0.1, lr=0.02, coef=None, out=BF, ranks=2, align=16, groups=None, calls=1):
    plan = Z.zero_plan(numels, ranks, align, groups)
    total = Z.zero_plan_info(plan)["psi_pad"]
    g = torch.Generator().manual_seed(sum(numels) + rows)
    master, momentum, reduced = (torch.randn(total, generator=g) * s for s in (0.02, 1e-3, 4e-3))
    GUARD = 256
    bufs = [torch.full((total + 2 * GUARD,), -77.0, device="cuda") for _ in range(3)]
    M, B, R = (b[GUARD:GUARD + total] for b in bufs)
    obuf = torch.full((total + 2 * GUARD,), -77.0, dtype=out, device="cuda")
    P = obuf[GUARD:GUARD + total]
    for t, v in ((M, master), (B, momentum), (R, reduced)):
        t.copy_(v)
    c = None if coef is None else torch.full((1,), coef, device="cuda")
    scale = 0.2 * math.sqrt(max(rows, cols))
    hp = Z.muon_hp(lr=lr, momentum=mu, weight_decay=wd, grad_scale=0.25, nesterov=nesterov, scale=scale)
    size = Z.zero_muon_workspace(rows, cols, len(tensors))
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    f = lambda v: torch.tensor(v, dtype=F32)  # noqa: E731
    rate, decay = f(lr) * f(scale), f(lr) * f(wd)
    want = master.double()
    allowed = {t: 0.0 for t in tensors}
    for _ in range(calls):
        Z.zero_muon_step(plan, tensors, rows, cols, M, B, R, hp, c, P, code(Z, out), work, size)
        for t in tensors:
            at = Z.zero_plan_tensor(plan, t)[0]
            s = slice(at, at + rows * cols)
            grad = reduced[s] * f(0.25) * f(1.0 if coef is None else coef)
            momentum[s] = f(mu) * momentum[s] + grad
            u = grad + f(mu) * momentum[s] if nesterov else momentum[s]
            o, off = O.allowance(u.reshape(rows, cols))
            want[s] = want[s] * (1 - decay.double()) - rate.double() * o.reshape(-1)
            # the update's own error, its rounding to fp16, three roundings of the weight
            allowed[t] += rate.item() * (off + 2.0 ** -11 * o.norm()) + 3 * 2.0 ** -24 * want[s].norm()
    torch.cuda.synchronize()
    assert torch.equal(B.cpu(), momentum), "momentum"
    assert torch.equal(R.cpu(), reduced)
    got = M.cpu()
    touched = torch.zeros(total, dtype=torch.bool)
    for t in tensors:
        at = Z.zero_plan_tensor(plan, t)[0]
        s = slice(at, at + rows * cols)
        touched[s] = True
        assert (got[s].double() - want[s]).norm() <= allowed[t], f"tensor {t}"
    assert torch.equal(got[~touched], master[~touched])
    assert torch.equal(P.cpu()[touched], got[touched].to(out)) and bool((P.cpu()[~touched] == -77.0).all())
    for b in bufs + [obuf]:
        assert bool((b[:GUARD] == -77.0).all() and (b[-GUARD:] == -77.0).all())


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("rows,cols,between", [(64, 96, 96), (96, 64, 5), (33, 71, 7), (130, 40, 1), (1, 50, 3), (50, 1, 2), (257, 300, 11)])
def test_step_on_tensors_of_a_plan(cuda, Z, rows, cols, between, nesterov):
    """Tensors at any place of the flat arrays, biases between them left alone."""
    numels = [between] + [rows * cols, between] * 3
    muon_step(Z, numels, [1, 3, 5], rows, cols, nesterov=nesterov)
    muon_step(Z, numels, [5, 1], rows, cols, nesterov=nesterov, wd=0.0, coef=0.3, out=F32)
    muon_step(Z, numels, [3], rows, cols, nesterov=nesterov, mu=0.0, align=1, ranks=3, calls=3)


def test_step_across_layer_groups(cuda, Z):
    muon_step(Z, [100, 48 * 80, 80, 48 * 80, 48 * 80, 9], [1, 3, 4], 48, 80, groups=[0, 1, 1, 2, 2, 3], ranks=4)


def test_step_without_parameters_or_tensors(cuda, Z):
    plan = Z.zero_plan([64 * 64], 2, 16)
    bufs = [torch.randn(4096, device="cuda") for _ in range(3)]
    before = [b.clone() for b in bufs]
    Z.zero_muon_step(plan, [], 64, 64, *bufs, Z.muon_hp(lr=0.1), None, None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bufs, before))
    size = Z.zero_muon_workspace(64, 64, 1)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    Z.zero_muon_step(plan, [0], 64, 64, *bufs, Z.muon_hp(lr=0.1), None, None, Z.ZERO_BF16, work, size)
    torch.cuda.synchronize()
    assert not torch.equal(bufs[0], before[0])


# ------------------------------------------------- streams, graphs, repeats --
def test_same_bits_on_any_stream_and_from_a_graph(cuda, Z):
    m, n, batch = 300, 200, 3
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(batch, m, n, device="cuda", generator=g)
    a, b = (torch.zeros(batch, m, n, dtype=BF, device="cuda") for _ in range(2))
    size = Z.zero_orthogonalize_workspace(m, n, batch)
    work = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ns = Z.newton_schulz()
    call = lambda y, w: Z.zero_orthogonalize(x, n, m * n, Z.ZERO_F32, m, n, batch, ns, y, n, m * n, w, size)  # noqa: E731
    call(a, work[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(b, work[1])
    call(a, work[0])                     # two calls at once, each with its own workspace
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    b.zero_()
    with torch.cuda.graph(graph):
        call(b, work[1])
    for _ in range(3):
        x.mul_(-2.0)                     # an odd function of the direction alone
        graph.replay()
        call(a, work[0])
        torch.cuda.synchronize()
        assert torch.equal(a, b)
