"""4-bit matrices at the ends of fp32's range: maxima so small that the tensor's
scale meets its least value, blocks of zeros beside them, and the largest."""
import pytest
import torch

import fp4_reference as Q
import ops_reference as R
from test_gpu_fp4 import Packed, fmt
from test_gpu_ops import code

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LEAST = 2.0 ** -117
TOP = {BF: torch.finfo(BF).max, F32: torch.finfo(F32).max}


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_optimizer_device_gb300 as Z
    return Z


def matrix(rows, cols, top, dtype):
    """Normal values whose largest is `top`, a row and two blocks of zeros."""
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(rows + cols), dtype=Q.D)
    x[3] = 0.0
    x[5, 16:32] = 0.0
    x[16:32, 7] = 0.0
    x = (x * (top / x.abs().max())).to(dtype)
    assert not torch.isinf(x).any()
    return x


def tensor_scale(Z, x):
    g = torch.full((1,), -1.0, device="cuda")
    work = torch.empty(Z.ZERO_FP4_WORKSPACE, dtype=torch.uint8, device="cuda")
    Z.zero_fp4_tensor_scale(x, x.shape[1], code(Z, x.dtype), *x.shape, g, work, work.numel())
    return g


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("top", [1e-24, 1e-30, 1e-32, 1e-33, 1e-36, 1e-37, 1e-38, 3e-40, 1e-42, "largest"])
def test_nv_by_its_own_scale(cuda, Z, top, dtype):
    """Codes and scales by the definition with g = max(amax / 2688, 2^-117), in each direction alone and in both; no NaN comes back, nor out of a product."""
    rows, cols = 40, 40                                    # scale tiles that blocks do not fill
    x = matrix(rows, cols, TOP[dtype] if top == "largest" else top, dtype)
    X = x.cuda()
    g = tensor_scale(Z, X)
    want = Q.tensor_scale(x)
    want = torch.maximum(want, torch.tensor(LEAST, dtype=Q.D))
    assert g.item() == want.item()
    ref, ref_t = Q.quantise(x, "nv", want), Q.quantise(x.t(), "nv", want)
    f = fmt(Z, "nv")
    both = [Packed(Z, rows, cols, "nv", 0, g) for _ in range(2)]
    alone = [Packed(Z, rows, cols, "nv", 0, g) for _ in range(2)]
    Z.zero_fp4_quantize(X, cols, code(Z, dtype), rows, cols, f, both[0].mat, both[1].mat)
    Z.zero_fp4_quantize(X, cols, code(Z, dtype), rows, cols, f, alone[0].mat, None)
    Z.zero_fp4_quantize(X, cols, code(Z, dtype), rows, cols, f, None, alone[1].mat)
    for q in (both, alone):
        q[0].check(*ref[:2], "q")
        q[1].check(*ref_t[:2], "qt")
    for out in (BF, F32):
        y = torch.empty(rows, cols, dtype=out, device="cuda")
        Z.zero_fp4_dequantize(both[0].mat, rows, cols, f, y, cols, code(Z, out))
        assert torch.equal(y.cpu(), ref[2].to(F32).to(out)) and (top == "largest" or not bool(torch.isnan(y).any()))
    if top == "largest":
        return
    # a product with ordinary values, of few rows and of many
    w = torch.randn(300, cols, generator=torch.Generator().manual_seed(9))
    gw = Q.tensor_scale(w)
    cw, bw, vw = Q.quantise(w, "nv", gw)
    qw = Packed(Z, 300, cols, "nv", 0, gw.to(F32).reshape(1).cuda()).fill(cw, bw)
    vx = ref[2]
    for m in (5, rows):
        o = torch.empty(m, 300, device="cuda")
        Z.zero_fp4_linear(both[0].mat, qw.mat, f, m, 300, cols, None, o, 300, Z.ZERO_F32)
        y, _, err, _ = R.linear(vx[:m], vw, False)
        # g_x g_w may be a subnormal number, off by half of 2^-149, and so may the result
        whole, size = want.item() * gw.item(), vx[:m].abs() @ vw.abs().T
        gap = 2.0 ** -150 * (1 + size / whole)
        assert bool(((o.cpu().double() - y).abs() <= err + 2.0 ** -22 * y.abs() + gap).all())
        assert bool((o[3] == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("g", [1e-42, LEAST, 1.0, 1.2e35])
def test_zeros_have_no_scale_whatever_the_whole_has(cuda, Z, g, dtype):
    x = torch.zeros(33, 70, dtype=dtype, device="cuda")
    whole = torch.full((1,), g, device="cuda")
    q, qt = Packed(Z, 33, 70, "nv", 0, whole), Packed(Z, 70, 33, "nv", 0, whole)
    for a, b in ((q, qt), (q, None), (None, qt)):
        Z.zero_fp4_quantize(x, 70, code(Z, dtype), 33, 70, fmt(Z, "nv"), a and a.mat, b and b.mat)
        for p in (a, b):
            if p is not None:
                assert not bool(p.codes.any()) and not bool(p.scales.any())
                p.codes.fill_(1)
                p.scales.fill_(1)


@pytest.mark.parametrize("g", [LEAST, 2.0 ** -100, 2.0 ** 100, 2.0 ** 115])
def test_a_given_scale_at_the_ends(cuda, Z, g):
    """Values of every size under one g: beyond 6 * 448 g to the largest, below its least to zero."""
    r = torch.Generator().manual_seed(4)
    x = torch.randn(64, 96, generator=r) * torch.exp2(torch.randint(-14, 14, (64, 6), generator=r).float()).repeat_interleave(16, 1)
    x = (x.double() * g).clamp(-3e38, 3e38).to(F32)
    whole = torch.full((1,), g, device="cuda")
    q, qt = Packed(Z, 64, 96, "nv", 0, whole), Packed(Z, 96, 64, "nv", 0, whole)
    Z.zero_fp4_quantize(x.cuda(), 96, Z.ZERO_F32, 64, 96, fmt(Z, "nv"), q.mat, qt.mat)
    G = torch.tensor(g, dtype=Q.D)
    q.check(*Q.quantise(x, "nv", G)[:2], "q")
    qt.check(*Q.quantise(x.t(), "nv", G)[:2], "qt")


@pytest.mark.parametrize("m", [1, 5, 8, 200])
@pytest.mark.parametrize("form", ["up", "down", "mixed"])
def test_mx_scales_far_from_one_another(cuda, Z, m, form):
    """Blocks scaled by 2^e against 2^-e for e to 127, either operand having the large one: sums of multiples of 1/4 below 2^15, exact in fp32."""
    n, k = 130, 320
    g = torch.Generator().manual_seed(m)
    codes = [torch.randint(0, 16, (r, k), generator=g, dtype=torch.uint8) for r in (m, n)]
    far = torch.tensor([100, 117, 118, 119, 120, 123, 125, 126, 127, 127])
    sign = {"up": torch.ones(10), "down": -torch.ones(10), "mixed": torch.tensor([1, -1] * 5)}[form].int()
    byte = [(127 + s * sign * far).to(torch.uint8).expand(r, 10).contiguous() for r, s in ((m, 1), (n, -1))]
    x, w = (Packed(Z, r, k, "mx").fill(c, b) for r, c, b in zip((m, n), codes, byte))
    v = [Q.LEVELS[(c & 7).long()] * torch.where(c > 7, -1.0, 1.0) for c in codes]
    assert bool((v[0].abs() @ v[1].abs().T < 2 ** 22).all())      # (and every partial sum's quarters below 2^24)
    y = torch.empty(m, n, device="cuda")
    Z.zero_fp4_linear(x.mat, w.mat, Z.ZERO_FP4_MX, m, n, k, None, y, n, Z.ZERO_F32)
    assert torch.equal(y.cpu().double(), v[0] @ v[1].T)


@pytest.mark.parametrize("m", [4, 200])
def test_mx_nan_beside_far_scales(cuda, Z, m):
    """A block whose scale is NaN makes its row NaN whatever the other operand's scale is."""
    n, k = 40, 64
    x, w = torch.full((m, k), 2, dtype=torch.uint8), torch.full((n, k), 2, dtype=torch.uint8)
    bx, bw = torch.full((m, 2), 127, dtype=torch.uint8), torch.full((n, 2), 127, dtype=torch.uint8)
    bx[2, 1], bw[7, 0], bw[9] = 255, 255, 254
    qx, qw = Packed(Z, m, k, "mx").fill(x, bx), Packed(Z, n, k, "mx").fill(w, bw)
    y = torch.empty(m, n, device="cuda")
    Z.zero_fp4_linear(qx.mat, qw.mat, Z.ZERO_FP4_MX, m, n, k, None, y, n, Z.ZERO_F32)
    want = torch.full((m, n), 64.0)
    want[:, 9] = float("inf")
    want[2], want[:, 7] = float("nan"), float("nan")
    y = y.cpu()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y, nan=0.0, posinf=-1.0), torch.nan_to_num(want, nan=0.0, posinf=-1.0))
