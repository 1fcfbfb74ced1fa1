"""Stage-3 training of GPT-2-style feed-forward sublayers, every kernel the
library's own.

Each sublayer is a layer group of a stage-3 plan: its bf16 parameters live as N
owner shards and are gathered before use (zero_gather_layer), computed with
(layer norm, product + GELU, product + dropout + residual, and their
gradients), and updated from the N ranks' gradients (zero_step_group).  The
ranks are emulated: N batches and N gradient buffers on one GPU.

    h' = h + dropout(gelu(norm(h) W1 + b1) W2 + b2)

    python examples/feed_forward_stage3.py --width 256 --layers 3 --ranks 4 --steps 30
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_optimizer_device_gb300 as Z  # noqa: E402

BF16 = torch.bfloat16
NAMES = ("norm_w", "norm_b", "fc_w", "fc_b", "proj_w", "proj_b")


def shapes(d: int) -> dict:
    """A sublayer's tensors in state-dict order, weights as GPT-2 keeps them."""
    return dict(zip(NAMES, ((d,), (d,), (d, 4 * d), (4 * d,), (4 * d, d), (d,))))


def tensors(flat: torch.Tensor, d: int) -> dict:
    """A group's flat buffer (parameters or gradients) as its tensors."""
    out, at = {}, 0
    for name, shape in shapes(d).items():
        n = shape[0] * (shape[1] if len(shape) > 1 else 1)
        out[name] = flat[at:at + n].view(shape)
        at += n
    return out


@dataclass
class Saved:
    """What a sublayer's backward pass needs of its forward pass."""
    h: torch.Tensor
    u: torch.Tensor
    z: torch.Tensor
    a: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor
    rng: object


def forward(p: dict, h: torch.Tensor, rng) -> tuple[torch.Tensor, Saved]:
    m, d = h.shape
    f = 4 * d
    u, z, a, y = (torch.empty(m, w, dtype=BF16, device=h.device) for w in (d, f, f, d))
    mean, rstd = (torch.empty(m, device=h.device) for _ in range(2))
    B = Z.ZERO_BF16
    Z.zero_layer_norm(h, d, B, p["norm_w"], p["norm_b"], B, m, d, Z.ZERO_NORM_LAYER, 1e-5, u, d, B,
                      mean, rstd)
    Z.zero_linear(u, d, p["fc_w"], f, Z.ZERO_W_KN, m, f, d,
                  Z.linear_epilogue(bias=p["fc_b"], act=Z.ZERO_ACT_GELU_TANH, pre=z, ldpre=f), a, f)
    Z.zero_linear(a, f, p["proj_w"], d, Z.ZERO_W_KN, m, d, f,
                  Z.linear_epilogue(bias=p["proj_b"], residual=h, ldres=d, dropout=rng), y, d)
    return y, Saved(h, u, z, a, mean, rstd, rng)


def backward(p: dict, g: dict, s: Saved, dy: torch.Tensor, add: bool,
             scratch: torch.Tensor) -> torch.Tensor:
    """Parameter gradients into g (added to what it holds if `add`); returns
    the gradient of h."""
    m, d = s.h.shape
    f = 4 * d
    B, KN = Z.ZERO_BF16, Z.ZERO_W_KN
    dd, dz, du, dh = (torch.empty(m, w, dtype=BF16, device=dy.device) for w in (d, f, d, d))
    Z.zero_dropout(dy, d, B, None, 0, B, m, d, s.rng, dd, d, B)
    Z.zero_linear_dweight(dd, d, s.a, f, m, d, f, KN, g["proj_w"], d, B, g["proj_b"], B, add)
    Z.zero_linear_dinput(dd, d, p["proj_w"], d, KN, m, d, f,
                         Z.linear_act_grad(Z.ZERO_ACT_GELU_TANH, s.z, f), dz, f)
    Z.zero_linear_dweight(dz, f, s.u, d, m, f, d, KN, g["fc_w"], f, B, g["fc_b"], B, add)
    Z.zero_linear_dinput(dz, f, p["fc_w"], f, KN, m, f, d, None, du, d)
    Z.zero_layer_norm_backward(du, d, B, s.h, d, B, p["norm_w"], B, s.mean, s.rstd, m, d,
                               Z.ZERO_NORM_LAYER, dy, d, dh, d, B, g["norm_w"], g["norm_b"], B, add,
                               scratch, Z.zero_layer_norm_workspace(m, d))
    return dh


def train(width: int = 256, layers: int = 3, ranks: int = 4, tokens: int = 512, steps: int = 30,
          dropout: float = 0.1, lr: float = 3e-3, seed: int = 0, report=None) -> list[float]:
    """Fits the sublayers to random targets; returns the loss of every step."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    sizes = [int(torch.Size(s).numel()) for s in shapes(width).values()]
    plan = Z.zero_plan(sizes * layers, ranks, 16, [ell for ell in range(layers) for _ in sizes])
    info = Z.zero_plan_info(plan)
    groups = [Z.zero_plan_group(plan, ell) for ell in range(layers)]
    master = torch.zeros(info["psi_pad"], device=dev)
    for grp in groups:
        p = tensors(master[grp["flat_off"]:grp["flat_off"] + grp["psi"]], width)
        p["norm_w"].fill_(1.0)
        p["fc_w"].normal_(0, 0.02, generator=gen)
        p["proj_w"].normal_(0, 0.02, generator=gen)
    moments = [torch.zeros_like(master) for _ in range(2)]
    full = master.to(BF16)
    shards = [torch.zeros(info["shard_total"], dtype=BF16, device=dev) for _ in range(ranks)]
    for grp in groups:                      # the owners' first bf16 shards
        for r in range(ranks):
            at = grp["flat_off"] + r * grp["shard"]
            shards[r][grp["rank_off"]:grp["rank_off"] + grp["shard"]] = full[at:at + grp["shard"]]
    layer = [torch.zeros(grp["psi_pad"], dtype=BF16, device=dev) for grp in groups]
    grads = [[torch.zeros(grp["psi_pad"], dtype=BF16, device=dev) for _ in range(ranks)] for grp in groups]
    scratch = torch.empty(max(16, Z.zero_layer_norm_workspace(tokens, width)), dtype=torch.uint8, device=dev)
    x = [torch.randn(tokens, width, device=dev, generator=gen).to(BF16) for _ in range(ranks)]
    target = [torch.randn(tokens, width, device=dev, generator=gen) for _ in range(ranks)]
    losses = []
    for step in range(1, steps + 1):
        loss = torch.zeros((), device=dev)
        # forward: gather a layer, use it for every rank's batch, go on
        h, saved = list(x), [[None] * ranks for _ in range(layers)]
        for ell in range(layers):
            Z.zero_gather_layer(plan, ell, shards, Z.ZERO_BF16, layer[ell])
            p = tensors(layer[ell], width)
            for r in range(ranks):
                rng = Z.dropout_rng(dropout, seed, (step * layers + ell) * ranks + r)
                h[r], saved[ell][r] = forward(p, h[r], rng)
        d = []
        for r in range(ranks):
            e = h[r].float() - target[r]
            loss += e.square().mean() / ranks
            d.append((e * (2.0 / width)).to(BF16))       # per token, as a model's loss is
        # backward: the same the other way round, a step per group
        hp = Z.adam_hp(step=step, grad_scale=1.0 / (ranks * tokens), lr=lr)
        for ell in reversed(range(layers)):
            Z.zero_gather_layer(plan, ell, shards, Z.ZERO_BF16, layer[ell])
            p = tensors(layer[ell], width)
            for r in range(ranks):
                d[r] = backward(p, tensors(grads[ell][r], width), saved[ell][r], d[r], False, scratch)
            Z.zero_step_group(plan, ell, grads[ell], Z.ZERO_BF16, master, *moments, hp, None, shards)
        losses.append(loss.item())
        if report:
            report(f"step {step:3d}  loss {losses[-1]:.4f}")
    return losses


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("width", 256), ("layers", 3), ("ranks", 4), ("tokens", 512), ("steps", 30)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--dropout", type=float, default=0.1)
    ap.add_argument("--lr", type=float, default=3e-3)
    train(**vars(ap.parse_args()), report=print)


if __name__ == "__main__":
    main()
