"""The layer operators where the order of things decides: boxes that land late,
operands shifted by two CTAs, calls side by side and back to back.  Results
are compared with 64 bits and, again and again with a cold cache, with
themselves: no bit may differ."""
import pytest
import torch

import ops_reference as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_optimizer_device_gb300 as Z
    return Z


@pytest.fixture(scope="module")
def flush():
    """Writes more than the L2 holds, so that the next call's operands come
    from memory."""
    junk = torch.empty(64 << 20, device="cuda")
    return lambda v: junk.fill_(v)


def rnd(seed, *shape, scale=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def product_bound(a, b, extra):
    """a @ b.T in 64 bits and what k fp32 terms in any order may miss of it."""
    a, b = a.to(R.D), b.to(R.D)
    return a @ b.T, (a.shape[1] + 4) * R.U32 * (a.abs() @ b.abs().T + extra)


def within(got, want, err, what):
    u = R.U16 if got.dtype == BF else R.U32
    bad = (got.to(R.D) - want).abs() > err + u * (want.abs() + err) + 1e-37
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} elements outside their bound"


# tiles 256 and 128 wide, whole and with an odd number of 32-column chunks
BOXES = [(4096, 4096, 512), (2048, 2504, 704), (1100, 3304, 1000), (2100, 2024, 2304)]


@pytest.mark.parametrize("m,n,k", BOXES)
def test_fp32_boxes_with_a_cold_residual(cuda, Z, flush, m, n, k):
    x, w, r = rnd(1, m, k), rnd(2, n, k, scale=k ** -0.5), rnd(3, m, n, dtype=F32)
    want, err = product_bound(x, w, r.to(R.D).abs())
    first = None
    for i in range(6):
        y = torch.full((m, n), -7.0, device="cuda")
        flush(i)
        ep = Z.linear_epilogue(residual=r, ldres=n, res_dtype=Z.ZERO_F32)
        Z.zero_linear(x, k, w, k, Z.ZERO_W_NK, m, n, k, ep, y, n, Z.ZERO_F32)
        if first is None:
            within(y, want + r.to(R.D), err, "y")
            first = y
        assert torch.equal(y, first), f"run {i} differs"


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("n,k,m", [(4096, 4096, 512), (2048, 2504, 704), (2504, 2104, 2304)])
def test_fp32_boxes_accumulating(cuda, Z, flush, n, k, m, kn):
    dy, x = rnd(1, m, n), rnd(2, m, k)
    shape = (k, n) if kn else (n, k)
    dw0 = rnd(3, *shape, dtype=F32)
    a, b = (x, dy) if kn else (dy, x)
    want, err = product_bound(a.T, b.T, dw0.to(R.D).abs())
    first = None
    for i in range(6):
        dw = dw0.clone()
        flush(i)
        Z.zero_linear_dweight(dy, n, x, k, m, n, k, Z.ZERO_W_KN if kn else Z.ZERO_W_NK, dw,
                              shape[1], Z.ZERO_F32, None, Z.ZERO_F32, True)
        if first is None:
            within(dw, want + dw0.to(R.D), err, "dw")
            first = dw
        assert torch.equal(dw, first), f"run {i} differs"


@pytest.mark.parametrize("m,n,k", BOXES)
def test_fp32_boxes_with_a_gate_and_kept_inputs(cuda, Z, flush, m, n, k):
    """Two slots a chunk, so two chunks in the ring: a tile with an odd number
    of chunks swaps the slots of the two sets of warps."""
    x, w, u = rnd(1, m, k), rnd(2, n, k, scale=k ** -0.5), rnd(3, m, n)
    z64, err = product_bound(x, w, 0)
    gate = u.to(R.D)
    first = None
    for i in range(6):
        y, z = torch.full((m, n), -7.0, device="cuda"), torch.full((m, n), -7.0, dtype=BF, device="cuda")
        flush(i)
        ep = Z.linear_epilogue(pre=z, ldpre=n, gate=u, ldgate=n)
        Z.zero_linear(x, k, w, k, Z.ZERO_W_NK, m, n, k, ep, y, n, Z.ZERO_F32)
        if first is None:
            within(z, z64, err, "pre")
            within(y, z64 * gate, err * gate.abs(), "y")
            first = y, z
        assert torch.equal(y, first[0]) and torch.equal(z, first[1]), f"run {i} differs"


# both operands off 16-byte boundaries, either one, rows along and across the contraction
SHIFTED = [(700, 1000, 1601, 1, 1), (700, 1000, 1600, 1, 0), (700, 1000, 1600, 0, 1),
           (2500, 3000, 515, 3, 5), (90, 520, 4099, 1, 1)]


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("m,n,k,pad_x,pad_w", SHIFTED)
def test_shifted_operands_with_a_cold_cache(cuda, Z, flush, m, n, k, pad_x, pad_w, kn):
    """A pair's second CTA shifts its part of a stage into place and the first
    one's tensor-core instructions read it: every stage must have arrived."""
    x = rnd(1, m, k + pad_x)[:, :k]
    w = rnd(2, *((k, n + pad_w) if kn else (n, k + pad_w)), scale=k ** -0.5)[:, :n if kn else k]
    want, err = product_bound(x, w.T if kn else w, 0)
    first = None
    for i in range(6):
        y = torch.full((m, n), -7.0, device="cuda")
        flush(i)
        Z.zero_linear(x, x.stride(0), w, w.stride(0), Z.ZERO_W_KN if kn else Z.ZERO_W_NK, m, n, k,
                      None, y, n, Z.ZERO_F32)
        if first is None:
            within(y, want, err, "y")
            first = y
        assert torch.equal(y, first), f"run {i} differs"


def test_products_side_by_side_on_two_streams(cuda, Z):
    """Calls that share the GPU and come in any order give the bits that each
    gives alone: aligned and shifted operands, split contractions, few rows."""
    sizes = [(2048, 2048, 1024, 0), (700, 1000, 1601, 1), (96, 512, 4096, 0), (5, 2048, 2048, 0),
             (1500, 777, 333, 3), (3000, 2056, 520, 0)]
    calls = []
    for i, (m, n, k, pad) in enumerate(sizes):
        x, w = rnd(i, m, k + pad)[:, :k], rnd(i + 50, n, k + pad, scale=k ** -0.5)[:, :k]

        def call(y, x=x, w=w, m=m, n=n, k=k):
            Z.zero_linear(x, x.stride(0), w, w.stride(0), Z.ZERO_W_NK, m, n, k, None, y, n, Z.ZERO_F32)
        alone = torch.empty(m, n, device="cuda")
        call(alone)
        calls.append((call, alone))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for s, order in zip(streams, (calls, calls[::-1])):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(4):
                for call, alone in order:
                    y = torch.full_like(alone, -7.0)
                    call(y)
                    outs.append((y, alone))
    torch.cuda.synchronize()
    for y, alone in outs:
        assert torch.equal(y, alone)


def layer_plan(Z, width, layers, ranks):
    """A plan of `layers` groups (norm weight, norm bias, product) and a way
    to give every owner its shard of a flat buffer."""
    sizes = [width, width, width * width]
    plan = Z.zero_plan(sizes * layers, ranks, 16, [ell for ell in range(layers) for _ in sizes])
    info, groups = Z.zero_plan_info(plan), [Z.zero_plan_group(plan, ell) for ell in range(layers)]
    shards = [torch.zeros(info["shard_total"], dtype=BF, device="cuda") for _ in range(ranks)]

    def give(full):
        for g in groups:
            for r in range(ranks):
                at = g["flat_off"] + r * g["shard"]
                shards[r][g["rank_off"]:g["rank_off"] + g["shard"]] = full[at:at + g["shard"]]
    return plan, info, groups, shards, give


@pytest.mark.parametrize("width", [256, 1000])
def test_gathers_and_their_readers_on_one_buffer_in_a_graph(cuda, Z, width):
    """Gather, norm, product, gather, norm, product on ONE layer buffer, in a
    replayed graph and straight on the stream: every reader starts while the
    gather before it still writes, and must see that gather's values; the
    next gather must not overtake a reader.  Between replays the shards
    change."""
    layers, ranks, m = 4, 3, 96
    plan, info, groups, shards, give = layer_plan(Z, width, layers, ranks)
    layer = torch.zeros(max(g["psi_pad"] for g in groups), dtype=BF, device="cuda")
    x = rnd(1, m, width)
    u = [torch.empty(m, width, dtype=BF, device="cuda") for _ in range(layers)]
    y = [torch.empty(m, width, device="cuda") for _ in range(layers)]
    du, dw = torch.empty_like(u[0]), torch.empty(layers, width, device="cuda")
    rstd = torch.empty(m, device="cuda")
    size = Z.zero_layer_norm_workspace(m, width)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    dx = [torch.empty(m, width, device="cuda") for _ in range(layers)]
    parts = lambda f: (f[:width], f[width:2 * width], f[2 * width:2 * width + width ** 2].view(width, width))  # noqa: E731

    def step():
        for ell in range(layers):
            Z.zero_gather_layer(plan, ell, shards, Z.ZERO_BF16, layer)
            nw, nb, w = parts(layer)
            Z.zero_layer_norm(x, width, 1, nw, nb, 1, m, width, Z.ZERO_NORM_RMS, 1e-5, u[ell], width, 1,
                              None, rstd)
            Z.zero_linear(u[ell], width, w, width, Z.ZERO_W_NK, m, width, width, None, y[ell], width,
                          Z.ZERO_F32)
            Z.zero_layer_norm_backward(u[ell], width, 1, x, width, 1, nw, 1, None, rstd, m, width,
                                       Z.ZERO_NORM_RMS, None, 0, dx[ell], width, 0, dw[ell], None, 0,
                                       False, work, size)

    def check(full):
        for ell, g in enumerate(groups):
            nw, nb, w = parts(full[g["flat_off"]:])
            r = (x.double().square().mean(1, keepdim=True) + 1e-5).rsqrt()
            h = x.double() * r
            want = h * nw.double() + nb.double()
            rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()  # noqa: E731
            assert rel(u[ell], want) < R.U16
            got = u[ell].double()
            assert rel(y[ell], got @ w.double().T) < 1e-5
            gw = got * nw.double()
            assert rel(dx[ell], r * (gw - h * (gw * h).mean(1, keepdim=True))) < 1e-4
            assert rel(dw[ell], (got * h).sum(0)) < 1e-4

    full = rnd(5, info["psi_pad"])
    give(full)
    step()
    check(full)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in range(5):
        full = rnd(10 + i, info["psi_pad"])
        give(full)
        graph.replay()
        if i % 2:
            graph.replay()           # back to back: the first gather follows the last reader
        check(full)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,width", [(64, 512), (3000, 1024)])
def test_norms_between_gathers(cuda, Z, m, width, dtype):
    """Gather, norm, gather, norm on one buffer and nothing between: a norm is
    resident while the one before it still reads the buffer's former values,
    and must not find those in its caches."""
    layers, ranks = 6, 2
    plan = Z.zero_plan([width, width] * layers, ranks, 16, [ell for ell in range(layers) for _ in range(2)])
    info, groups = Z.zero_plan_info(plan), [Z.zero_plan_group(plan, ell) for ell in range(layers)]
    code = Z.ZERO_BF16 if dtype == BF else Z.ZERO_F32
    shards = [torch.zeros(info["shard_total"], dtype=dtype, device="cuda") for _ in range(ranks)]
    layer = torch.zeros(max(g["psi_pad"] for g in groups), dtype=dtype, device="cuda")
    x = torch.ones(m, width, dtype=BF, device="cuda")          # normalises to 1: y = weight + bias
    x[:, 1::2] = -1
    y = [torch.empty(m, width, device="cuda") for _ in range(layers)]

    def step():
        for ell in range(layers):
            Z.zero_gather_layer(plan, ell, shards, code, layer)
            Z.zero_layer_norm(x, width, 1, layer[:width], layer[width:2 * width], code, m, width,
                              Z.ZERO_NORM_RMS, 0.0, y[ell], width, Z.ZERO_F32)

    step()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        step()
        step()
    for i in range(20):
        full = rnd(i, info["psi_pad"], dtype=dtype)
        for g in groups:
            for r in range(ranks):
                at = g["flat_off"] + r * g["shard"]
                shards[r][g["rank_off"]:g["rank_off"] + g["shard"]] = full[at:at + g["shard"]]
        graph.replay()
        for ell, g in enumerate(groups):
            w, b = (full[g["flat_off"] + o:g["flat_off"] + o + width].float() for o in (0, width))
            want = x.float() * w + b
            assert (y[ell] - want).abs().max().item() <= 4 * R.U32 * 8, (i, ell)
