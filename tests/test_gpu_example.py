"""The feed-forward example on the GPU: a sublayer's output and every gradient
against 64-bit autograd of its formulas, and a short training run."""
import os
import sys

import pytest
import torch

import ops_reference as R

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("tokens,width", [(1, 32), (77, 64), (300, 96), (260, 50)])
def test_sublayer_against_autograd(cuda, tokens, width):
    import feed_forward_stage3 as E
    Z = E.Z
    g = torch.Generator().manual_seed(tokens)
    flat = torch.cat([torch.randn(torch.Size(s).numel(), generator=g) * (0.1 if len(s) == 1 else s[0] ** -0.5) +
                      (1.0 if n == "norm_w" else 0.0) for n, s in E.shapes(width).items()]).to(E.BF16)
    h, dy = (torch.randn(tokens, width, generator=g).to(E.BF16) for _ in range(2))
    rng = Z.dropout_rng(0.2, 77, 5)
    pd = E.tensors(flat.cuda(), width)
    y, saved = E.forward(pd, h.cuda(), rng)
    grads = torch.zeros_like(flat).cuda()
    scratch = torch.empty(Z.zero_layer_norm_workspace(tokens, width), dtype=torch.uint8, device="cuda")
    dh = E.backward(pd, E.tensors(grads, width), saved, dy.cuda(), False, scratch)

    D = R.D
    p = {k: v.to(D).requires_grad_() for k, v in E.tensors(flat, width).items()}
    hd = h.to(D).requires_grad_()
    u = torch.nn.functional.layer_norm(hd, (width,), p["norm_w"], p["norm_b"], 1e-5)
    a = torch.nn.functional.gelu(u @ p["fc_w"] + p["fc_b"], approximate="tanh")
    keep = R.keep_mask(tokens, width, 0.2, 77, 5)
    want = hd + (a @ p["proj_w"] + p["proj_b"]) * keep / (1.0 - float(torch.tensor(0.2)))
    want.backward(dy.to(D))

    # six bf16 roundings lie between the inputs and the furthest gradient, each
    # 2^-9 of a value at most in the mean, and each product averages them
    tol = 6 * 2.0 ** -8
    rel = lambda x, w: ((x.cpu().to(D) - w).norm() / w.norm().clamp_min(1e-30)).item()  # noqa: E731
    assert rel(y, want.detach()) < tol
    assert rel(dh, hd.grad) < tol
    for name, t in E.tensors(grads, width).items():
        assert rel(t, p[name].grad) < tol, name


def test_training_reduces_the_loss(cuda):
    """Random targets of variance 1 from inputs of variance 1: the loss starts
    near 2 and falls; the same seed gives the same losses."""
    import feed_forward_stage3 as E
    a = E.train(width=64, layers=2, ranks=3, tokens=96, steps=25)
    assert 1.5 < a[0] < 2.5 and a[-1] < 0.9 * a[0]
    assert a == E.train(width=64, layers=2, ranks=3, tokens=96, steps=25)
