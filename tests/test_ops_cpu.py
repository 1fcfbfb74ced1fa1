"""CPU checks of the layer operators: the reference's random words against
published ones, its gradients against differences, every argument check (fake
addresses, never dereferenced), and the binding's checks of tensors."""
import ctypes

import numpy as np
import pytest
import torch

import ops_reference as R

Z = pytest.importorskip("zero_sharded_optimizer_device_gb300")
A = 1 << 40


def test_philox_known_answers():
    """The counter-based generator's published test vectors (Random123's
    kat_vectors for philox4x32-10)."""
    f = 0xFFFFFFFF
    for ctr, key, want in [
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((f, f, f, f), (f, f), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]:
        assert tuple(int(v) for v in R.philox(ctr, key)) == want


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9])
def test_keep_rate(p):
    """The mask keeps 1 - p of 40 000 elements within 5 standard deviations,
    and offsets give unrelated masks."""
    a, b = R.keep_mask(100, 400, p, 7, 0), R.keep_mask(100, 400, p, 7, 1)
    sd = (p * (1 - p) / 40000) ** 0.5
    assert abs(a.double().mean().item() - (1 - p)) <= 5 * sd + 1e-12
    both = (a & b).double().mean().item()
    assert abs(both - (1 - p) ** 2) <= 5 * ((1 - p) ** 2 * (1 - (1 - p) ** 2) / 40000) ** 0.5 + 1e-12


def _differences(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("name", R.ACTS)
def test_reference_activation_slopes(name):
    z = torch.linspace(-6, 6, 97, dtype=R.D) + 0.013
    got = _differences(lambda t: R.act(t, name)[0], z, torch.ones_like(z))
    assert (got - R.act(z, name)[1]).abs().max() < 1e-8


@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("name", R.ACTS)
def test_reference_linear_gradients(name, kn):
    """dinput through the activation and gate that made the input, and
    dweight, against central differences of the forward formulas."""
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=R.D)  # noqa: E731
    m, n, k = 5, 4, 6
    z, u, w, c = rn(m, k), rn(m, k), rn(*((k, n) if kn else (n, k))), rn(m, n)
    x = R.act(z, name)[0] * u
    loss = lambda z, u, w: (c * (R.act(z, name)[0] * u @ R.weight(w, kn))).sum()  # noqa: E731
    dx, dg, _, _ = R.linear_dinput(c, w, kn, name, z, u)
    dw, db, _, _ = R.linear_dweight(c, x, kn)
    for grad, arg in ((dx, 0), (dg, 1), (dw, 2)):
        args = [z, u, w]
        d = rn(*args[arg].shape)
        got = _differences(lambda t: loss(*[t if i == arg else a for i, a in enumerate(args)]),
                           args[arg], d)
        assert abs(got - (grad * d).sum()) < 1e-6
    assert torch.allclose(db, c.sum(0))


@pytest.mark.parametrize("rms", [False, True])
def test_reference_norm_gradients(rms):
    g = torch.Generator().manual_seed(4)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=R.D)  # noqa: E731
    x, w, b, c = rn(5, 9) + 0.5, rn(9), rn(9), rn(5, 9)
    y, mean, rstd, _ = R.norm(x, w, b, rms, 1e-5)
    dx, dw, db, _, _, _ = R.norm_backward(c, x, w, mean, rstd, rms)
    loss = lambda x, w, b: (c * R.norm(x, w, b, rms, 1e-5)[0]).sum()  # noqa: E731
    for grad, arg in ((dx, 0), (dw, 1), (db, 2)):
        args = [x, w, b]
        d = rn(*args[arg].shape)
        got = _differences(lambda t: loss(*[t if i == arg else a for i, a in enumerate(args)]),
                           args[arg], d)
        assert abs(got - (grad * d).sum()) < 1e-6


# ---------------------------------------------------------------- refusals --
def status(fn, *a, **k):
    with pytest.raises(Z.ZeroError) as e:
        fn(*a, stream=0, **k)
    return e.value.status


def lin(x=A, ldx=64, w=A + 64, ldw=64, layout=0, m=4, n=32, k=64, ep=None, y=A + 128, ldy=32,
        ydtype=1):
    return status(Z.zero_linear, x, ldx, w, ldw, layout, m, n, k, ep, y, ldy, ydtype)


@pytest.mark.parametrize("change,want", [
    (dict(x=None), "EINVAL"), (dict(w=0), "EINVAL"), (dict(y=None), "EINVAL"),
    (dict(m=-1), "EINVAL"), (dict(n=-1), "EINVAL"), (dict(k=-2), "EINVAL"),
    (dict(ldx=63), "EINVAL"), (dict(ldw=63), "EINVAL"), (dict(ldy=31), "EINVAL"),
    (dict(layout=2), "EINVAL"), (dict(layout=1, ldw=31), "EINVAL"),
    (dict(y=A), "EINVAL"), (dict(y=A + 64), "EINVAL"),
    (dict(x=A + 1), "EALIGN"), (dict(w=A + 65), "EALIGN"), (dict(y=A + 129), "EALIGN"),
    (dict(y=A + 130, ydtype=0), "EALIGN"), (dict(ydtype=2), "EDTYPE"),
    (dict(m=2 ** 31), "ERANGE"), (dict(ldx=2 ** 31), "ERANGE"), (dict(k=2 ** 31, ldx=2 ** 31), "ERANGE"),
])
def test_linear_refusals(change, want):
    assert lin(**change) == getattr(Z, "ZERO_" + want)


@pytest.mark.parametrize("ep,want", [
    (dict(act=5), "EINVAL"), (dict(act=-1), "EINVAL"),
    (dict(bias=A + 1), "EALIGN"), (dict(bias=A + 256, bias_dtype=3), "EDTYPE"),
    (dict(pre=A + 256, ldpre=31), "EINVAL"), (dict(pre=A, ldpre=32), "EINVAL"),
    (dict(pre=A + 128, ldpre=32), "EINVAL"), (dict(gate=A + 257, ldgate=32), "EALIGN"),
    (dict(gate=A + 128, ldgate=32), "EINVAL"), (dict(residual=A + 256, ldres=3), "EINVAL"),
    (dict(residual=A + 128, ldres=40), "EINVAL"),
    (dict(residual=A + 128, ldres=32, res_dtype=0), "EINVAL"),
    (dict(residual=A + 256, ldres=32, res_dtype=9), "EDTYPE"),
    (dict(dropout=Z.dropout_rng(-0.1, 0)), "EINVAL"), (dict(dropout=Z.dropout_rng(1.5, 0)), "EINVAL"),
    (dict(dropout=Z.dropout_rng(float("nan"), 0)), "EINVAL"),
    (dict(dropout=Z.dropout_rng(0.1, 0, 0, A + 4)), "EALIGN"),
])
def test_linear_epilogue_refusals(ep, want):
    assert lin(ep=Z.linear_epilogue(**ep)) == getattr(Z, "ZERO_" + want)


def test_linear_gradient_refusals():
    E = Z
    dinput = lambda ag=None, dx=A + 128, lddx=64, dt=1, m=4: status(  # noqa: E731
        Z.zero_linear_dinput, A, 32, A + 64, 64, 0, m, 32, 64, ag, dx, lddx, dt)
    assert dinput(dx=A) == E.ZERO_EINVAL and dinput(dx=None) == E.ZERO_EINVAL
    assert dinput(lddx=63) == E.ZERO_EINVAL and dinput(dt=5) == E.ZERO_EDTYPE
    assert dinput(m=2 ** 31) == E.ZERO_ERANGE
    ag = Z.linear_act_grad
    assert dinput(ag(2, None, 64)) == E.ZERO_EINVAL
    assert dinput(ag(7, A + 256, 64)) == E.ZERO_EINVAL
    assert dinput(ag(2, A + 256, 64, dgate=A + 512, lddgate=64)) == E.ZERO_EINVAL
    assert dinput(ag(2, A + 256, 64, gate=A + 512, ldgate=64, dgate=A + 512, lddgate=64)) == E.ZERO_EINVAL
    assert dinput(ag(2, A + 256, 64, gate=A + 513, ldgate=64)) == E.ZERO_EALIGN
    dweight = lambda dw=A + 128, lddw=64, dt=1, db=None, bt=1, layout=0: status(  # noqa: E731
        Z.zero_linear_dweight, A, 32, A + 64, 64, 4, 32, 64, layout, dw, lddw, dt, db, bt, 0)
    assert dweight(dw=A) == E.ZERO_EINVAL and dweight(dw=A + 64) == E.ZERO_EINVAL
    assert dweight(lddw=63) == E.ZERO_EINVAL and dweight(layout=1, lddw=31) == E.ZERO_EINVAL
    assert dweight(layout=9) == E.ZERO_EINVAL and dweight(dt=4) == E.ZERO_EDTYPE
    assert dweight(db=A + 128) == E.ZERO_EINVAL and dweight(db=A + 513) == E.ZERO_EALIGN
    assert dweight(db=A + 512, bt=2) == E.ZERO_EDTYPE


def test_dropout_refusals():
    rng = Z.dropout_rng(0.1, 1)
    d = lambda x=A, ldx=32, xt=1, r=None, ldr=0, rt=1, m=4, n=32, g=rng, y=A + 64, ldy=32, yt=1: \
        status(Z.zero_dropout, x, ldx, xt, r, ldr, rt, m, n, g, y, ldy, yt)  # noqa: E731
    assert d(x=None) == Z.ZERO_EINVAL and d(y=0) == Z.ZERO_EINVAL
    assert d(ldx=31) == Z.ZERO_EINVAL and d(n=-1) == Z.ZERO_EINVAL
    assert d(xt=2) == Z.ZERO_EDTYPE and d(y=A + 65) == Z.ZERO_EALIGN
    assert d(y=A, ldy=40) == Z.ZERO_EINVAL and d(y=A, yt=0) == Z.ZERO_EINVAL
    assert d(r=A + 64, ldr=40) == Z.ZERO_EINVAL and d(r=A + 128, ldr=3) == Z.ZERO_EINVAL
    assert d(g=Z.dropout_rng(2.0, 1)) == Z.ZERO_EINVAL
    assert d(m=2 ** 31) == Z.ZERO_ERANGE
    lib = Z.binding._lib()
    assert lib.zero_dropout(A, 32, 1, None, 0, 1, 4, 32, None, A + 64, 32, 1, None) == Z.ZERO_EINVAL
    bad = Z.dropout_rng(0.1, 1)
    bad.reserved = 1
    assert d(g=bad) == Z.ZERO_EINVAL


def test_layer_norm_refusals():
    f = lambda x=A, ldx=32, w=A + 512, b=None, pt=1, kind=0, eps=1e-5, y=A + 64, ldy=32, yt=1, \
        mean=None, rstd=None, m=4: status(Z.zero_layer_norm, x, ldx, 1, w, b, pt, m, 32, kind, eps,
                                          y, ldy, yt, mean, rstd)  # noqa: E731
    assert f(x=None) == Z.ZERO_EINVAL and f(w=None) == Z.ZERO_EINVAL and f(kind=2) == Z.ZERO_EINVAL
    assert f(eps=-1.0) == Z.ZERO_EINVAL and f(eps=float("inf")) == Z.ZERO_EINVAL
    assert f(eps=float("nan")) == Z.ZERO_EINVAL and f(pt=7) == Z.ZERO_EDTYPE
    assert f(kind=1, mean=A + 1024) == Z.ZERO_EINVAL and f(rstd=A + 1026) == Z.ZERO_EALIGN
    assert f(y=A, ldy=48) == Z.ZERO_EINVAL and f(b=A + 513) == Z.ZERO_EALIGN
    assert f(m=2 ** 31) == Z.ZERO_ERANGE
    need = Z.zero_layer_norm_workspace(4, 32)
    assert need >= 4 * 2 * 32
    g = lambda dy=A, x=A + 64, w=A + 512, mean=A + 1024, rstd=A + 2048, kind=0, dres=None, lddres=0, \
        dx=A + 128, lddx=32, dw=A + 4096, db=A + 8192, gt=1, ws=A + 65536, wb=need: status(
            Z.zero_layer_norm_backward, dy, 32, 1, x, 32, 1, w, 1, mean, rstd, 4, 32, kind, dres,
            lddres, dx, lddx, 1, dw, db, gt, 0, ws, wb)  # noqa: E731
    assert g(dy=None) == Z.ZERO_EINVAL and g(mean=None) == Z.ZERO_EINVAL
    assert g(rstd=None) == Z.ZERO_EINVAL and g(kind=1) == Z.ZERO_EINVAL
    assert g(dx=A) == Z.ZERO_EINVAL and g(dx=A + 64) == Z.ZERO_EINVAL
    assert g(dres=A + 128, lddres=40) == Z.ZERO_EINVAL and g(db=A + 4096) == Z.ZERO_EINVAL
    assert g(ws=None) == Z.ZERO_EINVAL and g(wb=need - 1) == Z.ZERO_EINVAL
    assert g(ws=A + 8) == Z.ZERO_EALIGN and g(gt=5) == Z.ZERO_EDTYPE and g(dw=None) == Z.ZERO_EINVAL
    out = ctypes.c_int64()
    lib = Z.binding._lib()
    assert lib.zero_layer_norm_workspace(-1, 4, ctypes.byref(out)) == Z.ZERO_EINVAL
    assert lib.zero_layer_norm_workspace(1, 4, None) == Z.ZERO_EINVAL
    assert lib.zero_layer_norm_workspace(1, 2 ** 31, ctypes.byref(out)) == Z.ZERO_ERANGE


def test_empty_outputs_need_no_device():
    """Calls that have nothing to write succeed without a launch."""
    Z.zero_linear(None, 64, A, 64, 0, 0, 32, 64, None, None, 32, 1, stream=0)
    Z.zero_linear_dinput(None, 32, A, 64, 0, 0, 32, 64, None, None, 64, 1, stream=0)
    Z.zero_dropout(None, 0, 1, None, 0, 1, 4, 0, Z.dropout_rng(0.5, 1), None, 0, 1, stream=0)
    Z.zero_layer_norm(None, 32, 1, A, None, 1, 0, 32, 0, 1e-5, None, 32, 1, stream=0)


def test_binding_refuses_wrong_tensors():
    bf, f32 = torch.zeros(64, dtype=torch.bfloat16), torch.zeros(64)
    with pytest.raises(ValueError, match="x: holds"):
        Z.zero_linear(bf, 16, A, 16, 0, 5, 8, 16, None, A + 64, 8, 1, stream=0)
    with pytest.raises(ValueError, match="x: a torch.float32"):
        Z.zero_linear(f32, 16, A, 16, 0, 4, 8, 16, None, A + 64, 8, 1, stream=0)
    with pytest.raises(ValueError, match="bias: holds"):
        Z.zero_linear(A, 16, A + 64, 16, 0, 4, 65, 16, Z.linear_epilogue(bias=bf), A + 128, 65, 1, stream=0)
    with pytest.raises(ValueError, match="w: holds"):
        Z.zero_linear_dinput(A, 8, bf[8:], 16, 0, 4, 4, 16, None, A + 64, 16, 1, stream=0)
    with pytest.raises(ValueError, match="dbias: a torch.bfloat16"):
        Z.zero_linear_dweight(A, 8, A + 64, 16, 4, 8, 16, 0, A + 128, 16, 1, bf, 0, 0, stream=0)
    with pytest.raises(ValueError, match="y: holds"):
        Z.zero_dropout(A, 16, 0, None, 0, 0, 4, 17, Z.dropout_rng(0.5, 1), f32, 17, 0, stream=0)
    with pytest.raises(ValueError, match="workspace: holds"):
        Z.zero_layer_norm_backward(A, 8, 1, A, 8, 1, A, 1, A, A, 4, 8, 0, None, 0, A, 8, 1, A, A, 1,
                                   0, f32, 257, stream=0)
    assert np.dtype(np.uint64).itemsize == 8
