"""4-bit products of long contractions on tensor cores, whose sums are not rounded to
nearest: results in bf16 up to and beyond the length from which sums are taken
out, and in fp32, of terms of one sign and of both."""
import pytest
import torch

import fp4_reference as Q
from test_gpu_fp4 import Packed, fmt
from test_gpu_ops import code

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_optimizer_device_gb300 as Z
    return Z


def operand(Z, g, rows, cols, form, one_sign):
    """Random codes under random scales, so that sums need more digits than fp32 has."""
    shape = (rows, -(-cols // Q.SIZE[form]))
    c = torch.randint(0, 8 if one_sign else 16, (rows, cols), generator=g, dtype=torch.uint8)
    s = (torch.randint(121, 128, shape, generator=g) if form == "mx" else torch.randint(40, 64, shape, generator=g)).to(torch.uint8)
    d = Q.E4M3[s.long()] if form == "nv" else torch.ldexp(torch.ones(shape, dtype=Q.D), s.int() - 127)
    v = Q.LEVELS[(c & 7).long()] * torch.where(c > 7, -1.0, 1.0) * d.repeat_interleave(Q.SIZE[form], 1)[:, :cols]
    return Packed(Z, rows, cols, form).fill(c, s), v.cuda()


@pytest.mark.parametrize("one_sign", [True, False], ids=["one", "both"])
@pytest.mark.parametrize("form", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", [(40, 300, 100001), (128, 512, 131072), (130, 264, 131100), (300, 260, 98304)])
def test_long_sums(cuda, Z, m, n, k, form, one_sign):
    g = torch.Generator().manual_seed(m + k)
    (x, vx), (w, vw) = operand(Z, g, m, k, form, one_sign), operand(Z, g, n, k, form, one_sign)
    want = vx @ vw.T
    share = lambda y: ((y * want).sum() / (want * want).sum()).item()  # noqa: E731
    for out in (BF, F32):
        y = torch.empty(m, n, dtype=out, device="cuda")
        Z.zero_fp4_linear(x.mat, w.mat, fmt(Z, form), m, n, k, None, y, n, code(Z, out))
        y = y.double()
        error = ((y - want).norm() / want.norm()).item()
        if out == F32:
            # 48 additions a round, each leaving off half a unit of the running sum on average, and 86 to nearest
            assert error < 2.9e-6
        else:
            # at most 2048 additions without rounding, each up to a unit (2^-23) of a sum that grows evenly: 2^-23 * 2048 / 2 of it, which is 2^-13; and the rounding to
            # bf16, at most 2^-8 of a value, whose share over all values is taken off (values next to a border leave some 1e-5)
            rounded = want.float().to(BF).double()
            assert error < 2.0 ** -8 + 2.0 ** -13 and abs(share(y) - share(rounded)) < 2.0 ** -13 + 2e-5
