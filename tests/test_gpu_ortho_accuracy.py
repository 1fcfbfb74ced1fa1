"""Orthogonalised updates against 64 bits without bf16's rounding: the step from
weights of zero, with lr = scale = 1, leaves the iteration's result in fp32
(rounded to fp16)."""
import pytest
import torch

import ortho_reference as O

pytestmark = pytest.mark.gpu
F32, D = torch.float32, torch.float64


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_optimizer_device_gb300 as Z
    return Z


def result(Z, xs, steps=5, coef=O.JORDAN):
    """The iteration's result of each matrix of xs [batch, m, n], on the GPU."""
    batch, m, n = xs.shape
    plan = Z.zero_plan([m * n] * batch, 1, 16)
    total = Z.zero_plan_info(plan)["psi_pad"]
    master, momentum, reduced = (torch.zeros(total, device="cuda") for _ in range(3))
    at = [Z.zero_plan_tensor(plan, t)[0] for t in range(batch)]
    for t in range(batch):
        reduced[at[t]:at[t] + m * n] = xs[t].reshape(-1)
    size = Z.zero_muon_workspace(m, n, batch)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    hp = Z.muon_hp(lr=1.0, momentum=0.0, nesterov=False, ns=Z.newton_schulz(steps, coef, 1e-7))
    Z.zero_muon_step(plan, list(range(batch)), m, n, master, momentum, reduced, hp, None, None, Z.ZERO_BF16, work, size)
    return [-master[a:a + m * n].view(m, n).to(D) for a in at]


def off(Z, xs, steps=5, coef=O.JORDAN):
    """The largest error of a batch, and the share by which results are too small (negative) or large."""
    worst, bias = 0.0, 0.0
    for x, got in zip(xs, result(Z, xs, steps, coef)):
        want = O.exact(x, steps, coef)
        worst = max(worst, ((got - want).norm() / want.norm()).item())
        share = ((got * want).sum() / (want * want).sum()).item() - 1
        bias = share if abs(share) > abs(bias) else bias
    return worst, bias


def random(batch, m, n, seed=0):
    return torch.randn(batch, m, n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


def steep(batch, m, n, seed=0):
    """Some strong directions over noise."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = min(m, n, 48)
    new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return torch.bmm(new(batch, m, r) * torch.arange(1, r + 1, device="cuda").float().pow(-0.7), new(batch, r, n)) + 0.5 * new(batch, m, n)


LONG = [(1, 64, 524288), (1, 524288, 64), (1, 2000003, 32), (2, 96, 50257), (3, 40000, 300), (3, 300, 40000), (5, 16385, 70), (5, 70, 16384), (2, 270, 32769)]


@pytest.mark.parametrize("batch,m,n", LONG)
def test_long_sides(cuda, Z, batch, m, n):
    """The accuracy that matrices of any length have.  Tensor cores leave 6e-9 of a sum of one sign off with every term, the diagonal of G: 3e-3 of it after 524288 if
    one accumulator takes them all, 1e-4 where sums are taken out every 16384.  With half of that to spare, and twice for G^2."""
    assert off(Z, random(batch, m, n), 1, (0.0, 1.0, 0.0))[1] == pytest.approx(0.0, abs=1.5e-4)
    assert off(Z, random(batch, m, n), 1, (0.0, 0.0, 1.0))[1] == pytest.approx(0.0, abs=3e-4)
    for x in (random(batch, m, n), steep(batch, m, n)):
        worst, bias = off(Z, x)
        assert worst < 1e-3 and abs(bias) < 3e-4


def test_the_same_bits_again(cuda, Z):
    """Several rounds in several tiles of each pair of CTAs."""
    x = random(24, 520, 33000)
    a, b = (torch.stack(result(Z, x, 2)) for _ in range(2))
    assert torch.equal(a, b)


# worst of 20 to 100 draws by the model of the number formats, rounded up; the result's rounding to fp16 is 2^-12 of it and adds in squares
MOST = ((12, 5e-3), (32, 2e-3), (257, 1.2e-3))
FULL = [(2, 64), (5, 64), (3, 8), (8, 8), (12, 40), (15, 15), (16, 256), (20, 20), (32, 32), (33, 71), (64, 64), (8192, 96), (128, 1024), (256, 256), (257, 300),
        (768, 768), (1024, 1024), (2048, 1536)]


def most(k):
    return next((bound for below, bound in MOST if k < below), 1.2e-3)


@pytest.mark.parametrize("m,n", FULL)
def test_full_rank(cuda, Z, m, n):
    assert off(Z, random(8 if m * n < 1 << 18 else 2, m, n, 1))[0] < most(min(m, n))


@pytest.mark.parametrize("m,n", [(5, 64), (8, 8), (40, 12), (16, 16), (16, 256), (500, 24), (32, 512), (64, 64), (64, 1024), (8192, 96), (96, 20000), (130, 128),
                                 (256, 1024), (1024, 255), (256, 256)])
def test_any_rank_of_a_smaller_side_to_256(cuda, Z, m, n):
    k = min(m, n)
    for r in sorted({1, 2, max(1, k // 8), max(1, k // 4), k // 2, k - 1}):
        xs = torch.bmm(random(4, m, r, 3 + r), random(4, r, n, 4 + r))
        assert off(Z, xs)[0] < most(k), f"rank {r}"


@pytest.mark.parametrize("m,n,rank,bound", [(257, 1024, 1, 2.5e-3), (257, 257, 32, 2.5e-3), (300, 257, 128, 2.5e-3), (768, 768, 1, 1.2e-3), (768, 768, 96, 1.2e-3),
                                            (768, 768, 384, 1.2e-3)])
def test_lower_rank_beyond(cuda, Z, m, n, rank, bound):
    xs = torch.bmm(random(4, m, rank, 3), random(4, rank, n, 4))
    assert off(Z, xs)[0] < bound


def test_a_batch_of_low_rank_and_long_sides(cuda, Z):
    """Parts of P and X and rounds of the Gram product together, more tiles than pairs of CTAs."""
    for x in (torch.bmm(random(12, 70, 3, 1), random(12, 3, 20011, 2)), torch.bmm(random(12, 20011, 3, 1), random(12, 3, 70, 2))):
        assert off(Z, x)[0] < 1.2e-3
        a, b = (torch.stack(result(Z, x)) for _ in range(2))
        assert torch.equal(a, b)


@pytest.mark.parametrize("m,n", [(16500, 16640), (16640, 16500)])
def test_rounds_of_every_product(cuda, Z, m, n):
    """Both sides beyond a round: some rows (columns of a tall x) of one step, each by products of vectors, y = a x + b G x + c G G x."""
    x = random(1, m, n, 5)[0]
    got = result(Z, x[None], 1)[0]
    (a, b, c), = O.coefficients(1)
    X = x.to(D) / (x.to(D).norm() + 1e-7)
    if m > n:
        X, got = X.T, got.T
    rows = [0, 1, 127, 255, 256, 4095, 16383, 16384, min(m, n) - 1]
    gram = lambda v: (v @ X) @ X.T  # noqa: E731
    e = torch.zeros(len(rows), X.shape[0], dtype=D, device="cuda")
    e[range(len(rows)), rows] = 1.0
    want = (a * e + b * gram(e) + c * gram(gram(e))) @ X
    y = got[rows]
    assert (y - want).norm() < 1e-3 * want.norm()
    assert ((y * want).sum() / (want * want).sum()).item() == pytest.approx(1.0, abs=3e-4)
