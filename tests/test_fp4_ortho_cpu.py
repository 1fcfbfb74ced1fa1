"""CPU checks of the 4-bit and the orthogonalising operators: their references
against hand values and each other, every argument check (fake addresses, never
dereferenced), the binding's checks of tensors, what their source may not hold."""
import ctypes
import os
import re

import pytest
import torch

import fp4_reference as Q
import ortho_reference as O

Z = pytest.importorskip("zero_sharded_optimizer_device_gb300")
A = 1 << 40
CSRC = os.path.join(os.path.dirname(Z.__file__), "csrc")


def status(fn, *a, **k):
    with pytest.raises(Z.ZeroError) as e:
        fn(*a, stream=0, **k)
    return e.value.name[5:]


# -------------------------------------------------------------- references --
def test_nearest_codes_by_hand():
    v = [0.0, 0.25, 0.26, 0.5, 0.75, 0.74, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 3.49, 5.0, 5.01, 6.0, 7.9, 1e30]
    want = [0, 0, 1, 1, 2, 1, 2, 3, 4, 4, 5, 6, 5, 6, 7, 7, 7, 7]
    assert Q.nearest_code(torch.tensor(v, dtype=Q.D)).tolist() == want


def test_nearest_scale_bytes():
    """Against torch's own E4M3 over all bytes, the places between two and beyond the last."""
    values = Q.E4M3
    assert torch.equal(values.float(), torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float())
    mid = (values[1:] + values[:-1]) / 2
    t = torch.cat([values, mid, mid * (1 + 1e-6), mid * (1 - 1e-6), torch.tensor([448.0, 500.0, 1e9], dtype=Q.D)])
    want = t.float().clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(Q.nearest_byte(Q.f32(t)), want)


def test_a_block_by_hand():
    x = torch.zeros(1, 40)
    x[0, :4] = torch.tensor([5.0, -2.6, 0.3, 9.0])        # amax 9: scale 2^(3 - 2) = 2
    x[0, 32] = 0.75                                        # a short block: scale 2^(-1 - 2)
    code, byte, v = Q.quantise(x, "mx")
    assert byte.tolist() == [[128, 124]]
    assert v[0, :4].tolist() == [4.0, -3.0, 0.0, 8.0] and v[0, 32] == 0.75   # 2.5, 1.3, .15, 4.5 go to 2, 1.5, 0, 4
    code, byte, v = Q.quantise(torch.tensor([[6.0, 3.0, -0.6] + [0.0] * 13]), "nv", torch.tensor(0.5))
    assert byte.tolist() == [[0x40]] and v[0, :3].tolist() == [6.0, 3.0, -0.5]     # amax / 3 = 2 = E4M3 0x40; d = 1
    packed, scales = Q.pack(code, byte, "nv")
    assert packed.shape == (1, 16) and packed[0, 0] == 0x57 and packed[0, 1] == 0x09 and scales.shape == (512,) and scales[0] == 0x40


def test_sizes():
    for form, code in (("mx", Z.ZERO_FP4_MX), ("nv", Z.ZERO_FP4_NV)):
        for rows, cols in ((0, 0), (1, 1), (128, 128), (129, 129), (5, 64), (300, 1000)):
            assert Z.zero_fp4_size(rows, cols, code) == Q.size(rows, cols, form)


def test_quantisation_error_of_normal_values():
    """Codes of 1 and more stand for x / scale from 0.75 on: off by at most half
    a step, largest against the value where 0.75 becomes 1 (1/3; 2.5 to 2 and 5
    to 4 are 1/5), or a quarter where 8 (the most before the next scale) becomes 6."""
    x = torch.randn(64, 256, generator=torch.Generator().manual_seed(1))
    for form, g in (("mx", None), ("nv", Q.tensor_scale(x))):
        code, byte, v = Q.quantise(x, form, g)
        big = (code & 7) >= 2
        assert ((v - x.double()).abs() / x.double().abs())[big].max() <= (1 + 1e-6) / 3


@pytest.mark.parametrize("m,n", [(6, 9), (9, 6), (5, 5)])
def test_steps_act_on_singular_values(m, n):
    x = torch.randn(m, n, generator=torch.Generator().manual_seed(2), dtype=O.D)
    y = O.exact(x, 3, eps=0.0)
    u, s, v = torch.linalg.svd(x, full_matrices=False)
    s = s / s.norm()
    for a, b, c in O.coefficients(3):
        s = a * s + b * s ** 3 + c * s ** 5
    assert (y - u @ torch.diag(s) @ v).abs().max() < 1e-12


def test_model_error_is_what_the_header_says():
    """Five steps with the kernels' number formats: 5e-4 to 1e-3 off, at any spectrum."""
    g = torch.Generator().manual_seed(3)
    for x in (torch.randn(256, 256, generator=g), torch.randn(100, 400, generator=g), torch.randn(256, 8, generator=g) @ torch.randn(8, 256, generator=g)):
        e = O.exact(x)
        assert (O.model(x) - e).norm() < 1.2e-3 * e.norm()


# ---------------------------------------------------------------- refusals --
def fp4(codes=A, ld=32, scales=A + 4096, g=None):
    return Z.fp4_matrix(codes, ld, scales, g)


@pytest.mark.parametrize("change,want", [
    (dict(x=None), "EINVAL"), (dict(ldx=63), "EINVAL"), (dict(xt=3), "EDTYPE"), (dict(x=A + 1), "EALIGN"), (dict(rows=-1), "EINVAL"), (dict(rows=2 ** 31), "ERANGE"),
    (dict(form=2), "EINVAL"), (dict(form=-1), "EINVAL"), (dict(q=None, qt=None), "EINVAL"), (dict(q=fp4(ld=16)), "EINVAL"), (dict(q=fp4(ld=40)), "EALIGN"),
    (dict(q=fp4(codes=A + 8)), "EALIGN"), (dict(q=fp4(scales=A + 4097)), "EALIGN"), (dict(q=fp4(codes=None)), "EINVAL"), (dict(q=fp4(scales=None)), "EINVAL"),
    (dict(q=fp4(ld=2 ** 31)), "ERANGE"), (dict(q=fp4(scales=A)), "EINVAL"), (dict(q=fp4(g=A + 64)), "EINVAL"), (dict(form=1, q=fp4(g=A + 66)), "EALIGN"),
    (dict(form=1, q=fp4(g=A + 64), qt=fp4(A + 8192, 16, A + 12288, A + 68)), "EINVAL"), (dict(qt=fp4(A + 8192, 16, A + 4096)), "EINVAL"),
    (dict(qt=fp4(A, 16, A + 12288)), "EINVAL"), (dict(q=fp4(codes=A + 65536)), "EINVAL"), (dict(qt=fp4(A + 8192, 16, A + 65536)), "EINVAL"),
])
def test_quantize_refusals(change, want):
    a = dict(x=A + 65536, ldx=64, xt=1, rows=8, cols=64, form=0, q=fp4(), qt=None)
    a.update(change)
    assert status(Z.zero_fp4_quantize, a["x"], a["ldx"], a["xt"], a["rows"], a["cols"], a["form"], a["q"], a["qt"]) == want


def test_dequantize_and_tensor_scale_refusals():
    d = lambda q=fp4(), form=0, y=A + 65536, ldy=64, yt=1, rows=8: status(Z.zero_fp4_dequantize, q, rows, 64, form, y, ldy, yt)  # noqa: E731
    assert d(form=7) == "EINVAL" and d(y=None) == "EINVAL" and d(y=A) == "EINVAL" and d(y=A + 4096) == "EINVAL" and d(ldy=63) == "EINVAL"
    assert d(yt=5) == "EDTYPE" and d(y=A + 65537) == "EALIGN" and d(q=fp4(g=A + 64)) == "EINVAL" and d(rows=2 ** 31) == "ERANGE"
    assert d(q=None) == "EINVAL"
    t = lambda x=A, g=A + 64, w=A + 4096, b=Z.ZERO_FP4_WORKSPACE, xt=1: status(Z.zero_fp4_tensor_scale, x, 64, xt, 8, 64, g, w, b)  # noqa: E731
    assert t(x=None) == "EINVAL" and t(g=None) == "EINVAL" and t(w=None) == "EINVAL" and t(b=4095) == "EINVAL" and t(g=A) == "EINVAL"
    assert t(w=A) == "EINVAL" and t(w=A + 64) == "EINVAL" and t(g=A + 66) == "EALIGN" and t(w=A + 4100) == "EALIGN" and t(xt=9) == "EDTYPE"
    lib, n = Z.binding._lib(), ctypes.c_int64()
    assert lib.zero_fp4_size(4, 4, 0, None, ctypes.byref(n)) == Z.ZERO_EINVAL and lib.zero_fp4_size(4, 4, 5, ctypes.byref(n), ctypes.byref(n)) == Z.ZERO_EINVAL
    assert lib.zero_fp4_size(-1, 4, 0, ctypes.byref(n), ctypes.byref(n)) == Z.ZERO_EINVAL and lib.zero_fp4_size(4, 2 ** 31, 0, ctypes.byref(n), ctypes.byref(n)) == Z.ZERO_ERANGE


def test_4_bit_product_refusals():
    x, w, y = fp4(A, 32, A + 4096), fp4(A + 8192, 32, A + 12288), A + 65536
    f = lambda x=x, w=w, form=0, m=8, n=40, k=64, ep=None, y=y, ldy=40, yt=1: status(Z.zero_fp4_linear, x, w, form, m, n, k, ep, y, ldy, yt)  # noqa: E731
    assert f(x=None) == "EINVAL" and f(w=None) == "EINVAL" and f(y=None) == "EINVAL" and f(form=3) == "EINVAL" and f(m=-1) == "EINVAL"
    assert f(k=65) == "EINVAL" and f(ldy=39) == "EINVAL" and f(yt=2) == "EDTYPE" and f(y=y + 1) == "EALIGN" and f(n=2 ** 31, ldy=2 ** 31) == "ERANGE"
    assert f(y=A) == "EINVAL" and f(y=A + 12288) == "EINVAL" and f(x=fp4(g=A + 64)) == "EINVAL"
    e = Z.linear_epilogue
    assert f(ep=e(act=9)) == "EINVAL" and f(ep=e(pre=A, ldpre=40)) == "EINVAL" and f(ep=e(pre=y, ldpre=40)) == "EINVAL" and f(ep=e(gate=y + 4097, ldgate=40)) == "EALIGN"
    assert f(ep=e(residual=y, ldres=48)) == "EINVAL" and f(ep=e(bias=y + 1)) == "EALIGN" and f(ep=e(dropout=Z.dropout_rng(2.0, 0))) == "EINVAL"
    d = lambda ag=None, dx=y, lddx=64, dt=1: status(Z.zero_fp4_linear_dinput, fp4(A, 32, A + 4096), fp4(A + 8192, 32, A + 12288), 0, 8, 40, 64, ag, dx, lddx, dt)  # noqa: E731
    g = Z.linear_act_grad
    assert d(dx=A + 8192) == "EINVAL" and d(lddx=63) == "EINVAL" and d(dt=4) == "EDTYPE" and d(g(2, None, 64)) == "EINVAL" and d(g(8, A + 1024, 64)) == "EINVAL"
    assert d(g(2, y + 4096, 64, gate=y + 8192, ldgate=64, dgate=A, lddgate=64)) == "EINVAL" and d(g(2, y, 64)) == "EINVAL"
    dw = lambda out=y, ld=64, dt=1, m=64: status(Z.zero_fp4_linear_dweight, fp4(A, 32, A + 4096), fp4(A + 8192, 32, A + 12288), 0, m, 40, 64, out, ld, dt)  # noqa: E731
    assert dw(out=None) == "EINVAL" and dw(out=A) == "EINVAL" and dw(ld=63) == "EINVAL" and dw(dt=7) == "EDTYPE" and dw(m=65) == "EINVAL"


def test_orthogonalize_refusals():
    need = Z.zero_orthogonalize_workspace(8, 16, 3)
    ns = Z.newton_schulz()
    f = lambda x=A, ldx=16, sx=128, xt=1, m=8, n=16, batch=3, ns=ns, y=A + 65536, ldy=16, sy=128, w=A + (1 << 20), b=need: status(  # noqa: E731
        Z.zero_orthogonalize, x, ldx, sx, xt, m, n, batch, ns, y, ldy, sy, w, b)
    assert f(x=None) == "EINVAL" and f(y=None) == "EINVAL" and f(w=None) == "EINVAL" and f(b=need - 1) == "EINVAL" and f(ns=None) == "EINVAL"
    assert f(ldx=15) == "EINVAL" and f(ldy=15) == "EINVAL" and f(sx=127) == "EINVAL" and f(sy=127) == "EINVAL" and f(m=-1) == "EINVAL" and f(batch=-1) == "EINVAL"
    assert f(xt=3) == "EDTYPE" and f(x=A + 1) == "EALIGN" and f(y=A + 65537) == "EALIGN" and f(w=A + 8) == "EALIGN"
    assert f(y=A, xt=0) == "EINVAL" and f(y=A, ldy=24, sy=192) == "EINVAL" and f(y=A, sy=256) == "EINVAL" and f(w=A) == "EINVAL"
    assert f(batch=65536) == "ERANGE" and f(m=2 ** 31) == "ERANGE" and f(m=2 ** 30, batch=3, sx=2 ** 35, sy=2 ** 35) == "ERANGE"
    for bad in (dict(steps=-1), dict(steps=17)):
        c = Z.zero_newton_schulz_t(**bad)
        assert f(ns=c) == "EINVAL"
    for eps, coef in ((-1.0, 1.0), (float("nan"), 1.0), (float("inf"), 1.0), (1e-7, float("nan")), (1e-7, float("inf"))):
        assert f(ns=Z.newton_schulz(2, (1.0, coef, 0.5), eps)) == "EINVAL"
    lib, out = Z.binding._lib(), ctypes.c_int64()
    assert lib.zero_orthogonalize_workspace(4, 4, 1, None) == Z.ZERO_EINVAL and lib.zero_muon_workspace(4, 4, 1, None) == Z.ZERO_EINVAL
    assert lib.zero_muon_workspace(4, 4, 129, ctypes.byref(out)) == Z.ZERO_ERANGE and lib.zero_muon_workspace(4, 4, -1, ctypes.byref(out)) == Z.ZERO_EINVAL
    with pytest.raises(ValueError, match="2 triples for 3 steps"):
        Z.newton_schulz(3, [(1, 2, 3), (4, 5, 6)])


def test_muon_step_refusals():
    plan = Z.zero_plan([128, 10, 128, 128, 0], 2, 16)
    need = Z.zero_muon_workspace(8, 16, 3)

    def f(tensors=(0, 2, 3), rows=8, cols=16, master=A, mom=A + 65536, red=A + 131072, coef=None, out=A + 196608, ot=1, w=A + (1 << 20), b=need, plan=plan, **hp):
        h = Z.muon_hp(**{**dict(lr=0.1), **{k: v for k, v in hp.items() if k != "reserved"}})
        h.reserved = hp.get("reserved", 0)
        return status(Z.zero_muon_step, plan, list(tensors), rows, cols, master, mom, red, h, coef, out, ot, w, b)

    assert f(tensors=(0, 1)) == "EINVAL" and f(tensors=(0, 4)) == "EINVAL" and f(tensors=(0, 5)) == "ERANGE" and f(tensors=(-1,)) == "ERANGE"
    assert f(tensors=(0, 2, 0)) == "EINVAL" and f(tensors=[0] * 129) == "ERANGE" and f(rows=16) == "EINVAL" and f(rows=-8) == "EINVAL"
    assert f(master=None) == "EINVAL" and f(mom=None) == "EINVAL" and f(red=None) == "EINVAL" and f(w=None) == "EINVAL" and f(b=need - 1) == "EINVAL"
    assert f(master=A + 4) == "EALIGN" and f(mom=A + 65540) == "EALIGN" and f(out=A + 196610) == "EALIGN" and f(coef=A + 2) == "EALIGN" and f(w=A + 8) == "EALIGN"
    assert f(ot=4) == "EDTYPE" and f(mom=A) == "EINVAL" and f(red=A) == "EINVAL" and f(out=A) == "EINVAL" and f(red=A + 65536) == "EINVAL" and f(w=A) == "EINVAL"
    assert f(lr=float("nan")) == "EINVAL" and f(momentum=1.0) == "EINVAL" and f(momentum=-0.1) == "EINVAL" and f(scale=float("inf")) == "EINVAL" and f(reserved=1) == "EINVAL"
    assert f(ns=Z.newton_schulz(2, (1.0, 2.0, 3.0), -1.0)) == "EINVAL"
    lib = Z.binding._lib()
    hp = Z.muon_hp(lr=0.1)
    t = (ctypes.c_int64 * 1)(0)
    call = lambda plan, t, n, hp: lib.zero_muon_step(plan, t, n, 8, 16, A, A + 65536, A + 131072, hp, None, None, 0, A + (1 << 20), need, None)  # noqa: E731
    assert call(None, t, 1, ctypes.byref(hp)) == Z.ZERO_EINVAL and call(plan, None, 1, ctypes.byref(hp)) == Z.ZERO_EINVAL
    assert call(plan, t, -1, ctypes.byref(hp)) == Z.ZERO_EINVAL and call(plan, t, 1, None) == Z.ZERO_EINVAL


def test_nothing_to_do_needs_no_device():
    Z.zero_fp4_quantize(None, 64, 1, 0, 64, 0, fp4(None, 32, None), stream=0)
    Z.zero_fp4_dequantize(fp4(None, 0, None), 8, 0, 0, None, 0, 1, stream=0)
    Z.zero_fp4_linear(fp4(None, 32, None), fp4(), 0, 0, 8, 64, None, None, 8, 1, stream=0)
    Z.zero_orthogonalize(None, 16, 0, 1, 0, 16, 1, Z.newton_schulz(), None, 16, 0, None, 0, stream=0)
    plan = Z.zero_plan([128], 2, 16)
    Z.zero_muon_step(plan, [], 8, 16, A, A + 65536, A + 131072, Z.muon_hp(lr=0.1), None, None, stream=0)


def test_binding_refuses_wrong_tensors():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    x, y = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16)
    big = u8(512)
    with pytest.raises(ValueError, match="q.codes: holds"):
        Z.zero_fp4_quantize(A, 64, 0, 4, 64, 0, Z.fp4_matrix(u8(4, 31), 32, big), stream=0)
    with pytest.raises(ValueError, match="q.scales: holds"):
        Z.zero_fp4_quantize(A, 64, 0, 4, 64, 0, Z.fp4_matrix(u8(4, 32), 32, u8(511)), stream=0)
    with pytest.raises(ValueError, match="qt.codes: holds"):
        Z.zero_fp4_quantize(A, 64, 0, 4, 64, 0, None, Z.fp4_matrix(u8(63, 16), 16, big), stream=0)
    with pytest.raises(ValueError, match="not consecutive"):
        Z.zero_fp4_dequantize(Z.fp4_matrix(u8(64, 64)[:, ::2], 64, big), 4, 64, 0, A, 64, stream=0)
    with pytest.raises(ValueError, match="tensor_scale: holds"):
        Z.zero_fp4_quantize(A, 64, 0, 4, 64, 1, Z.fp4_matrix(u8(4, 32), 32, big, u8(3)), stream=0)
    with pytest.raises(ValueError, match="x: a torch.float32"):
        Z.zero_fp4_tensor_scale(x, 64, 1, 4, 64, A, A + 4096, 4096, stream=0)
    with pytest.raises(ValueError, match="workspace: holds"):
        Z.zero_fp4_tensor_scale(A, 64, 1, 4, 64, A, big, 4096, stream=0)
    with pytest.raises(ValueError, match="y: holds"):
        Z.zero_orthogonalize(A, 64, 256, 1, 4, 64, 2, Z.newton_schulz(), y, 64, 256, A, 1 << 30, stream=0)
    with pytest.raises(ValueError, match="x: a torch.float32"):
        Z.zero_orthogonalize(x, 64, 256, 1, 4, 64, 1, Z.newton_schulz(), A, 64, 256, A, 1 << 30, stream=0)
    plan = Z.zero_plan([256], 2, 16)
    with pytest.raises(ValueError, match="momentum: holds"):
        Z.zero_muon_step(plan, [0], 4, 64, A, torch.zeros(255), A, Z.muon_hp(lr=0.1), None, None, 1, A, 1 << 30, stream=0)


# ------------------------------------------------------------------ source --
@pytest.mark.parametrize("name", ["zero_tile.cuh", "zero_product.cuh", "zero_walk.cuh", "zero_fp4.cuh", "zero_fp4.cu", "zero_fp4_rows.cu", "zero_ortho.cu"])
def test_kernels_that_start_early_load_coherently(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__ldg|\bld\.global(\.\w+)*\.nc\b|__restrict__|\bld_once\b", code)
    assert not re.search(r"__trap|\basm\b[^;]*\btrap;", code)
