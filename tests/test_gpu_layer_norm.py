"""Layer norm on the GPU, forward and backward, against its formulas in 64 bits.

Tolerances, with u = 2^-24 (half an fp32 step) and h half a step of the storage type: a sum of n values of which no
partial sum holds more than k additions is off by at most k u sum|value|. The kernels' chains are the pieces of a thread
(at most 8 x 8 values, or C / 64 where the strip is read again), 6 steps over the lanes, up to 16 over the waves: k = 200
covers the sizes below (C / 64 + 30 for the largest). With it
  mean:  k u mean|x|            (and u |mean|)
  rstd:  half of the variance's relative error, (k + 8) u
  y:     h |y| + |gamma| (k u mean|x| rstd + |xhat| (k + 8) u) + 4 u (|gamma xhat| + |beta|)
  dx:    h |dx| + rstd (k u (mean|g| + |xhat| mean|g xhat|) + 8 u (|g| + |mean g| + |xhat mean(g xhat)|))
  dgamma, dbeta: h |sum| + (k + 4) u sum|term|: a thread adds at most M / 64 terms here, below k
(the squares of these errors are below u times them). bf16: h = 2^-8 |value|, a whole half step of its 8 bits.
"""
import pytest
import torch

from ff_input_projection_amd import EALIAS, EALIGN, EINVAL, FusedProjError, FusedProjection, LayerNorm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
K = 200
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
B, F = torch.bfloat16, torch.float32

# (layout, dtype, batch, channels, spatial, pad)
CASES = [
    ("tokens_last", B, 3, 1, (5,), 0), ("tokens_last", F, 3, 1, (5,), 0), ("tokens_last", B, 1, 8, (1,), 0),
    ("tokens_last", B, 2, 7, (9,), 0), ("tokens_last", F, 2, 3, (9,), 1), ("tokens_last", B, 5, 320, (31,), 8),
    ("tokens_last", B, 2, 768, (129,), 0), ("tokens_last", B, 2, 769, (33,), 3), ("tokens_last", B, 3, 1387, (17,), 5),
    ("tokens_last", B, 2, 2048, (6,), 0), ("tokens_last", B, 2, 2056, (6,), 0), ("tokens_last", B, 16, 4096, (1,), 0),
    ("tokens_last", B, 2, 4099, (3,), 1), ("tokens_last", B, 1, 8192, (5,), 0), ("tokens_last", B, 1, 8193, (3,), 0),
    ("tokens_last", B, 2, 16385, (2,), 0), ("tokens_last", B, 1, 32768, (3,), 0),
    ("tokens_last", F, 2, 512, (40,), 0), ("tokens_last", F, 2, 1024, (9,), 0), ("tokens_last", F, 2, 1025, (9,), 2),
    ("tokens_last", F, 3, 2500, (5,), 0), ("tokens_last", F, 1, 4096, (7,), 0), ("tokens_last", F, 2, 4097, (3,), 0),
    ("tokens_last", F, 2, 9000, (3,), 0), ("tokens_last", F, 1, 16388, (3,), 0), ("tokens_last", F, 1, 32765, (2,), 3),
    ("channels_first", B, 2, 1, (3,), 0), ("channels_first", B, 1, 5, (1,), 0), ("channels_first", F, 2, 5, (7,), 0),
    ("channels_first", B, 2, 32, (8, 8, 1), 0), ("channels_first", B, 3, 320, (5, 13), 0),
    ("channels_first", B, 2, 768, (32, 4, 1), 0), ("channels_first", B, 2, 769, (67,), 3),
    ("channels_first", B, 2, 1030, (64,), 0), ("channels_first", B, 2, 1408, (72,), 0),
    ("channels_first", B, 1, 1537, (24,), 1), ("channels_first", B, 1, 2049, (31,), 0),
    ("channels_first", B, 1, 5000, (9,), 0), ("channels_first", F, 2, 320, (199,), 2),
    ("channels_first", F, 2, 600, (6, 6, 3), 0), ("channels_first", F, 1, 1100, (33,), 0),
    ("channels_first", F, 1, 1600, (32,), 0), ("channels_first", F, 2, 4200, (5,), 0),
    ("channels_first", B, 70, 24, (50,), 0), ("channels_first", F, 300, 9, (11,), 0), ("tokens_last", B, 700, 40, (3,), 0),
]
IDS = [f"{c[0][:2]}_{'bf16' if c[1] is B else 'f32'}_b{c[2]}_c{c[3]}_s{'x'.join(map(str, c[4]))}_pad{c[5]}" for c in CASES]


def make(layout, dtype, batch, channels, spatial, pad, seed=1, offset=3.0):
    """(x as a view with `pad` further channels between slabs or rows, gamma, beta, dy), on the GPU."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    if layout == "channels_first":
        x = r(batch, channels + pad, *spatial) * 1.7 + offset
        x = x.to(dtype).to(DEV)[:, :channels]
        dy = r(batch, channels, *spatial)
    else:
        x = r(batch, spatial[0], channels + pad) * 1.7 + offset
        x = x.to(dtype).to(DEV)[..., :channels]
        dy = r(batch, spatial[0], channels)
    gamma, beta = 1.0 + 0.3 * r(channels), 0.5 * r(channels)
    return x, gamma.to(dtype).to(DEV), beta.to(dtype).to(DEV), dy.to(dtype).to(DEV)


def rows(t, layout):
    """[tokens, channels] in 64 bits on the CPU."""
    t = t.double().cpu()
    return t.flatten(2).transpose(1, 2).reshape(-1, t.shape[1]) if layout == "channels_first" else t.reshape(-1, t.shape[2])


def check(name, got, want, tol):
    got = got.double().cpu()
    assert got.shape == want.shape, name
    assert torch.isfinite(got).all(), name
    err = (got - want).abs()
    print(f"[layer_norm] {name}: max err/tol {(err / tol.clamp(min=1e-300)).max().item():.3g}", flush=True)
    assert (err <= tol).all(), name   # both are 0 where a single channel leaves nothing


def forward_reference(x, gamma, beta, eps):
    mean = x.mean(1, keepdim=True)
    rstd = (((x - mean) ** 2).mean(1, keepdim=True) + eps) ** -0.5
    xhat = (x - mean) * rstd
    return xhat * gamma + beta, mean, rstd, xhat


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    print(f"[case] layer_norm forward {case}", flush=True)
    layout, dtype = case[0], case[1]
    x, gamma, beta, _ = make(*case)
    ln = LayerNorm.for_tensor(x, layout, eps=1e-3)
    y = torch.full(x.shape, float("nan"), dtype=dtype, device=DEV)
    stats = torch.full((2, ln.M), float("nan"), device=DEV)
    ln(x, gamma, beta, out=(y, stats))
    torch.cuda.synchronize()
    x64, g, b = rows(x, layout), gamma.double().cpu(), beta.double().cpu()
    y64, mean, rstd, xhat = forward_reference(x64, g, b, float(torch.tensor(1e-3, dtype=torch.float32)))
    spread = x64.abs().mean(1, keepdim=True)
    check("mean", stats[0], mean[:, 0], (K * U * spread + U * mean.abs())[:, 0])
    check("rstd", stats[1], rstd[:, 0], (rstd * (K + 8) * U)[:, 0])
    tol = HALF[dtype] * y64.abs() + g.abs() * (K * U * spread * rstd + xhat.abs() * (K + 8) * U)
    check("y", rows(y, layout), y64, tol + 4 * U * ((g * xhat).abs() + b.abs()))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    print(f"[case] layer_norm backward {case}", flush=True)
    layout, dtype = case[0], case[1]
    x, gamma, beta, dy = make(*case, seed=2, offset=0.3)
    ln = LayerNorm.for_tensor(x, layout, eps=1e-3)
    _, stats = ln(x, gamma, beta)
    nan = lambda s: torch.full(s, float("nan"), dtype=dtype, device=DEV)
    out = (nan(x.shape), nan((ln.C,)), nan((ln.C,)))
    workspace = torch.full((ln.workspace_bytes() // 4,), float("nan"), device=DEV)
    dx, dgamma, dbeta = ln.backward(x, gamma, stats, dy, out=out, workspace=workspace)
    torch.cuda.synchronize()
    x64, g, d = rows(x, layout), gamma.double().cpu(), rows(dy, layout)
    mean, rstd = (t[:, None] for t in stats.double().cpu())
    xhat, gd = (x64 - mean) * rstd, d * g
    c1, c2 = gd.mean(1, keepdim=True), (gd * xhat).mean(1, keepdim=True)
    want = rstd * (gd - c1 - xhat * c2)
    tol = K * U * (gd.abs().mean(1, keepdim=True) + xhat.abs() * (gd * xhat).abs().mean(1, keepdim=True))
    tol = tol + 8 * U * (gd.abs() + c1.abs() + (xhat * c2).abs())
    check("dx", rows(dx, layout), want, HALF[dtype] * want.abs() + rstd * tol)
    for name, got, terms in (("dgamma", dgamma, d * xhat), ("dbeta", dbeta, d)):
        want = terms.sum(0)
        check(name, got, want, HALF[dtype] * want.abs() + (K + 4) * U * terms.abs().sum(0))


def test_gradient_against_differences():
    """The gradients are the slopes of sum(y dy): central differences of the formula in 64 bits."""
    case = ("tokens_last", F, 2, 12, (3,), 0)
    x, gamma, beta, dy = make(*case, seed=5, offset=0.5)
    ln = LayerNorm.for_tensor(x, "tokens_last", eps=1e-2)
    _, stats = ln(x, gamma, beta)
    dx, dgamma, dbeta = (t.double().cpu() for t in ln.backward(x, gamma, stats, dy))
    x64, g, b, d = x.double().cpu(), gamma.double().cpu(), beta.double().cpu(), dy.double().cpu()

    def loss(x_, g_, b_):
        return float((forward_reference(x_.reshape(6, 12), g_, b_, 1e-2)[0] * d.reshape(6, 12)).sum())

    step = 1e-5   # the third derivative's share is about step^2 = 1e-10, the rounding's 1e-16 / 1e-5
    for at in ((0, 0, 0), (1, 2, 11), (0, 1, 5)):
        e = torch.zeros_like(x64)
        e[at] = step
        assert abs((loss(x64 + e, g, b) - loss(x64 - e, g, b)) / (2 * step) - float(dx[at])) < 1e-5
    for i in (0, 7):
        e = torch.zeros_like(g)
        e[i] = step
        assert abs((loss(x64, g + e, b) - loss(x64, g - e, b)) / (2 * step) - float(dgamma[i])) < 1e-5
        assert abs((loss(x64, g, b + e) - loss(x64, g, b - e)) / (2 * step) - float(dbeta[i])) < 1e-5


@pytest.mark.parametrize("layout", ["tokens_last", "channels_first"])
def test_far_from_zero(layout):
    """Values 1000 standard deviations from zero: the variance has no cancellation to lose."""
    case = (layout, F, 2, 300, (40,), 0)
    x, gamma, beta, _ = make(*case, offset=1700.0)
    ln = LayerNorm.for_tensor(x, layout)
    _, stats = ln(x, gamma, beta)
    x64 = rows(x, layout)
    _, mean, rstd, _ = forward_reference(x64, 1.0, 0.0, 1e-5)
    # the mean is off by up to K u 1700 = 2e-2 standard deviations' hundredth: its square is what the variance gets
    check("mean", stats[0], mean[:, 0], K * U * x64.abs().mean(1))
    check("rstd", stats[1], rstd[:, 0], rstd[:, 0] * ((K + 8) * U + (K * U * 1700 * rstd[:, 0]) ** 2))


@pytest.mark.parametrize("layout", ["tokens_last", "channels_first"])
@pytest.mark.parametrize("dtype", [B, F])
def test_non_finite_values_stay_with_their_token_and_channel(layout, dtype):
    x, gamma, beta, dy = make(layout, dtype, 2, 40, (24,), 0)
    ln = LayerNorm.for_tensor(x, layout)
    y0, s0 = ln(x, gamma, beta)
    g0 = ln.backward(x, gamma, s0, dy)
    bad = x.clone()
    at = (slice(None), 3, 7) if layout == "channels_first" else (slice(None), 7, 3)
    bad[(0,) + at[1:]] = float("nan")
    bad[(1,) + at[1:]] = float("inf")
    y, s = ln(bad, gamma, beta)
    hit = torch.zeros(48, dtype=torch.bool)
    hit[[7, 24 + 7]] = True
    a, b = rows(y, layout), rows(y0, layout)
    assert torch.isnan(a[hit]).all() and torch.equal(a[~hit], b[~hit])
    dx, dgamma, dbeta = ln.backward(bad, gamma, s, dy)
    a, b = rows(dx, layout), rows(g0[0], layout)
    assert torch.isnan(a[hit]).all() and torch.equal(a[~hit], b[~hit])
    assert torch.isnan(dgamma).all() and torch.equal(dbeta, g0[2])   # dbeta sums dy alone
    d = dy.clone()
    d[(0,) + at[1:]] = float("inf")
    dx, dgamma, dbeta = ln.backward(x, gamma, s0, d)
    a = rows(dx, layout)
    assert not torch.isfinite(a[7]).any() and torch.equal(a[~hit], b[~hit])
    one = torch.zeros(40, dtype=torch.bool)
    one[3] = True
    for got, was in ((dgamma, g0[1]), (dbeta, g0[2])):
        assert not torch.isfinite(got.cpu()[one]).any() and torch.equal(got.cpu()[~one], was.cpu()[~one])


def test_no_bias_no_stats_no_tokens():
    x, gamma, beta, dy = make("tokens_last", B, 2, 64, (5,), 0)
    with_bias, without = LayerNorm.for_tensor(x, "tokens_last"), LayerNorm.for_tensor(x, "tokens_last", has_bias=False)
    y, stats = without(x, gamma)
    zero, _ = with_bias(x, gamma, torch.zeros_like(beta))
    assert torch.equal(y, zero)
    y2 = torch.empty_like(y)
    assert without(x, gamma, out=(y2, None))[1] is None
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    dx, dgamma, dbeta = without.backward(x, gamma, stats, dy)
    want = with_bias.backward(x, gamma, stats, dy)
    assert dbeta is None and torch.equal(dx, want[0]) and torch.equal(dgamma, want[1])
    for shape in ((0, 5, 64), (2, 0, 64)):
        e = torch.empty(shape, dtype=B, device=DEV)
        ln = LayerNorm.for_tensor(e, "tokens_last")
        y, stats = ln(e, gamma, beta)
        assert y.shape == shape and stats.shape == (2, 0)
        dx, dgamma, dbeta = ln.backward(e, gamma, stats, e.contiguous())
        torch.cuda.synchronize()
        assert not dgamma.any() and not dbeta.any()


def test_one_slab_read_by_every_sequence():
    """A stride of 0 over the batch: x is read where it lies, y is dense."""
    one, gamma, beta, _ = make("tokens_last", F, 1, 96, (7,), 0)
    x = one.expand(4, 7, 96)
    y, _ = LayerNorm.for_tensor(x, "tokens_last")(x, gamma, beta)
    want, _ = LayerNorm.for_tensor(one, "tokens_last")(one, gamma, beta)
    assert y.is_contiguous() and torch.equal(y, want.expand(4, 7, 96))


def test_refusals():
    x, gamma, beta, dy = make("tokens_last", B, 2, 64, (5,), 0)
    ln = LayerNorm.for_tensor(x, "tokens_last")
    y, stats = ln(x, gamma, beta)
    lib, h, st = ln._lib, ln._h, torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr()
    assert lib.layer_norm_run(h, p(x), p(gamma), None, p(y), p(stats), st) == EINVAL
    assert lib.layer_norm_run(h, None, p(gamma), p(beta), p(y), p(stats), st) == EINVAL
    assert lib.layer_norm_run(h, p(x), p(gamma), p(beta), p(y) + 1, p(stats), st) == EALIGN
    assert lib.layer_norm_run(h, p(x), p(gamma), p(beta), p(y), p(stats) + 2, st) == EALIGN
    assert lib.layer_norm_run(h, p(x), p(gamma), p(beta), p(x), p(stats), st) == EALIAS
    assert lib.layer_norm_run(h, p(x), p(gamma), p(beta), p(y), p(y), st) == EALIAS
    ws = torch.empty(ln.workspace_bytes(), dtype=torch.uint8, device=DEV)
    grads = [torch.empty_like(t) for t in (x, gamma, beta)]
    args = [p(t) for t in (x, gamma, stats, dy, *grads, ws)]
    assert lib.layer_norm_backward(h, *args, ws.numel() - 4, st) == EINVAL
    for i in range(8):
        assert lib.layer_norm_backward(h, *args[:i], None, *args[i + 1:], ws.numel(), st) == EINVAL, i
    assert lib.layer_norm_backward(h, *args[:4], args[3], *args[5:], ws.numel(), st) == EALIAS
    assert lib.layer_norm_backward(h, *args[:5], args[6], *args[6:], ws.numel(), st) == EALIAS
    with pytest.raises(ValueError):
        ln(x[:, :4], gamma, beta)
    with pytest.raises(ValueError):
        ln(x, gamma)
    with pytest.raises(ValueError):
        ln(x, gamma[:32], beta)
    with pytest.raises(ValueError):
        ln(x, gamma.cpu(), beta)
    with pytest.raises(TypeError):
        ln(x.float().to(torch.float32), gamma, beta)
    with pytest.raises(ValueError):
        ln.backward(x, gamma, stats[:1], dy)
    with pytest.raises(ValueError):
        ln.backward(x, gamma, stats, dy.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(FusedProjError):
        ln.backward(x, gamma, stats, dy, workspace=ws[:16])
    torch.cuda.synchronize()


@pytest.mark.parametrize("layout", ["tokens_last", "channels_first"])
def test_graph_replays_streams_and_determinism(layout):
    """Captured forward and backward replay to the eager bits, with other work in between; two streams at once (a
    workspace each) give them too."""
    x, gamma, beta, dy = make(layout, B, 3, 200, (130,), 0)
    ln = LayerNorm.for_tensor(x, layout)
    y, stats = ln(x, gamma, beta)
    eager = [y, stats, *ln.backward(x, gamma, stats, dy)]
    eager = [t.clone() for t in eager]
    torch.cuda.synchronize()
    outs = [torch.empty_like(t) for t in eager]
    ws = torch.empty(ln.workspace_bytes(), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        ln(x, gamma, beta, out=outs[:2])
        ln.backward(x, gamma, outs[1], dy, out=outs[2:], workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        ln(x, gamma, beta)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in streams:
            y, stats = ln(x, gamma, beta, stream=s)
            got.append([y, stats, *ln.backward(x, gamma, stats, dy, stream=s)])
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, eager):
            assert torch.equal(a, b)


@pytest.mark.parametrize("layout", ["tokens_last", "channels_first"])
def test_norm_and_projection_in_training(layout):
    """x -> layer norm -> fused projection, and the gradients back through both, against 64-bit autograd.

    fp32 throughout: every value is off by at most some hundred u of the sums of magnitudes it is made of (C = 64 terms a
    product, 48 columns and 66 tokens in the gradients). 2000 u of the largest magnitude of each tensor is far above that
    and far below any wrong term."""
    tokens = (66,) if layout == "tokens_last" else (4, 33)
    x, gamma, beta, _ = make(layout, F, 2, 64, tokens, 0, seed=9)
    if layout == "channels_first":
        x = x[..., :32].contiguous()
    g = torch.Generator().manual_seed(3)
    w = (torch.randn((64, 48), generator=g) / 8).to(DEV)
    ln = LayerNorm.for_tensor(x, layout)
    proj = FusedProjection.for_tensor(torch.empty(x.shape, device=DEV), layout, ff_dim=24, ff_act="gelu", n_heads=2, head_dim=4)
    y, stats = ln(x, gamma, beta)
    ff, q, k, v = proj(y, w)
    ups = [torch.randn(t.shape, generator=g).to(DEV) for t in (ff, q, k, v)]
    dy, dw, _ = proj.backward(y, w, None, *ups)
    dx, dgamma, dbeta = ln.backward(x, gamma, stats, dy.view(x.shape))
    torch.cuda.synchronize()

    leaves = [t.double().cpu().requires_grad_() for t in (x, gamma, beta, w)]
    x64, g64, b64, w64 = leaves
    r = x64.flatten(2).transpose(1, 2).reshape(-1, 64) if layout == "channels_first" else x64.reshape(-1, 64)
    mean = r.mean(1, keepdim=True)
    n = (r - mean) * (((r - mean) ** 2).mean(1, keepdim=True) + 1e-5) ** -0.5 * g64 + b64
    z = n @ w64
    parts = [torch.nn.functional.gelu(z[:, :24]).view(ff.shape)]
    parts += [z[:, 24 + 8 * i:32 + 8 * i].view(2, -1, 2, 4).transpose(1, 2).reshape(q.shape) for i in range(3)]
    loss = sum((p * u.double().cpu()).sum() for p, u in zip(parts, ups))
    loss.backward()
    for name, got, want in [("ff", ff, parts[0].detach()), ("q", q, parts[1].detach()), ("dx", dx, x64.grad),
                            ("dgamma", dgamma, g64.grad), ("dbeta", dbeta, b64.grad), ("dw", dw, w64.grad)]:
        check(name, got, want, torch.full_like(want, 2000 * U * want.abs().max().item()))


@pytest.mark.parametrize("layout", ["tokens_last", "channels_first"])
def test_more_tokens_than_one_dimension_of_a_grid(layout):
    """1.2 million slabs of one token, and 5 million tokens: more workgroups than a grid's dimension takes at once."""
    batch, tokens = (1_200_000, 1) if layout == "channels_first" else (1, 5_000_000)
    shape = (batch, 8, tokens) if layout == "channels_first" else (batch, tokens, 8)
    g = torch.Generator(device=DEV).manual_seed(1)
    x, dy = (torch.randn(shape, generator=g, device=DEV) for _ in range(2))
    gamma, beta = torch.linspace(0.5, 1.5, 8, device=DEV), torch.linspace(-1.0, 1.0, 8, device=DEV)
    ln = LayerNorm.for_tensor(x, layout)
    y, stats = ln(x, gamma, beta)
    dx, dgamma, dbeta = ln.backward(x, gamma, stats, dy)
    torch.cuda.synchronize()
    axis, wide = (1, [1, 8, 1]) if layout == "channels_first" else (2, [1, 1, 8])
    x64, d = x.double(), dy.double()
    mean = x64.mean(axis, keepdim=True)
    rstd = ((x64 - mean).square().mean(axis, keepdim=True) + 1e-5) ** -0.5
    xhat, g64 = (x64 - mean) * rstd, gamma.double().view(wide)
    want = xhat * g64 + beta.double().view(wide)
    # sums of 8: at most 8 u of the mean magnitude each, and a rounding a step
    tol = 16 * U * (g64 * (x64.abs().mean(axis, keepdim=True) * rstd + xhat.abs()) + 1.0)
    assert ((y.double() - want).abs() <= tol).all()
    gd = d * g64
    want = rstd * (gd - gd.mean(axis, keepdim=True) - xhat * (gd * xhat).mean(axis, keepdim=True))
    # x - mean carries 10 u of |x| too, and the given statistics 16 u
    tol = 40 * U * rstd * (gd.abs() + gd.abs().mean(axis, keepdim=True) + (xhat.abs() + 1 + x64.abs() * rstd)
                           * (gd * xhat).abs().mean(axis, keepdim=True) * (1 + x64.abs().mean(axis, keepdim=True) * rstd))
    assert ((dx.double() - want).abs() <= tol).all()
    other = (0, 2) if layout == "channels_first" else (0, 1)
    for got, terms in ((dgamma, d * xhat), (dbeta, d)):
        # up to 5000 additions a thread: their roundings add up to 5000 u of the sum of magnitudes at most
        assert ((got.double() - terms.sum(other)).abs() <= 6000 * U * (terms.abs() + d.abs()).sum(other)).all()


def test_tensors_of_another_device_are_refused(monkeypatch):
    """A plan made where another device was current takes no tensors of this one, in either path."""
    x, gamma, beta, dy = make("tokens_last", B, 2, 64, (5,), 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    ln = LayerNorm.for_tensor(x, "tokens_last")
    monkeypatch.undo()
    with pytest.raises(ValueError):
        ln(x, gamma, beta)
    with pytest.raises(ValueError):
        ln(x, gamma, beta, out=(torch.empty_like(x), None))
    with pytest.raises(ValueError):
        ln.backward(x, gamma, torch.zeros((2, 10), device=DEV), dy)


# (layout, dtype, batch, channels, tokens): more strips or rows than twice the workgroups, the last turn of some of them only
TURNS = [
    # strips of 32 (bf16) or 16 tokens, 1024, 512 or 256 workgroups; slabs that end with a strip, and ones that do not
    ("channels_first", B, 70, 40, 1000), ("channels_first", B, 70, 40, 1024), ("channels_first", B, 70, 384, 1000),
    ("channels_first", F, 40, 200, 1000), ("channels_first", F, 40, 200, 1008), ("channels_first", F, 40, 384, 1001),
    ("channels_first", B, 40, 768, 1000), ("channels_first", B, 40, 700, 1024), ("channels_first", F, 20, 513, 1000),
    ("channels_first", B, 20, 1408, 1000), ("channels_first", B, 20, 1030, 1024), ("channels_first", F, 20, 800, 600),
    # more channels than a workgroup holds; slabs shorter than a strip
    ("channels_first", B, 20, 1600, 1000), ("channels_first", F, 12, 1700, 1008), ("channels_first", B, 700, 24, 11),
    # 8, 2 and 1 rows a workgroup, 512 of them
    ("tokens_last", B, 1, 40, 10001), ("tokens_last", B, 1, 2048, 9001), ("tokens_last", B, 3, 1387, 3001),
    ("tokens_last", F, 1, 1000, 9001), ("tokens_last", B, 1, 4096, 2501), ("tokens_last", B, 1, 4099, 2501),
    ("tokens_last", B, 1, 8192, 2100), ("tokens_last", F, 1, 1387, 2501), ("tokens_last", F, 1, 4096, 2501),
    ("tokens_last", B, 1, 8200, 1300), ("tokens_last", B, 1, 16385, 1100), ("tokens_last", F, 1, 4100, 1300),
    ("tokens_last", F, 1, 9000, 1100), ("tokens_last", F, 1, 20000, 1100),
]


@pytest.mark.parametrize("case", TURNS, ids=[f"{c[0][:2]}_{'bf16' if c[1] is B else 'f32'}_b{c[2]}_c{c[3]}_s{c[4]}" for c in TURNS])
def test_backward_of_workgroups_that_take_several_turns(case):
    """x, dy and the tokens' means are whole numbers, their rstds powers of two: every term of dgamma and dbeta is a multiple
    of a half below 2^7, and a thread adds fewer than 2^15 of them: below 2^23, every partial sum is exact in 24 bits. A
    strip or row that is lost, doubled or swapped shows in full."""
    print(f"[case] layer_norm turns {case}", flush=True)
    layout, dtype, batch, channels, tokens = case
    first = layout == "channels_first"
    g = torch.Generator(device=DEV).manual_seed(21)
    whole = lambda low, high, *s: torch.randint(low, high + 1, s, generator=g, device=DEV).to(torch.float64)
    shape = (batch, channels, tokens) if first else (batch, tokens, channels)
    x, dy = whole(-8, 8, *shape), whole(-4, 5, *shape)     # dy's mean is a half: whole turns weigh in
    mean, rstd = whole(-2, 3, batch, tokens), 2.0 ** whole(-1, 1, batch, tokens)
    gamma = (1.0 + 0.3 * torch.randn(channels, generator=g, device=DEV)).to(dtype)
    ln = LayerNorm(shape, torch.empty(shape, device="meta").stride(), layout, dtype)
    nan = lambda s: torch.full(s, float("nan"), dtype=dtype, device=DEV)
    out = (nan(shape), nan((channels,)), nan((channels,)))
    workspace = torch.full((ln.workspace_bytes() // 4,), float("nan"), device=DEV)
    stats = torch.stack([mean.reshape(-1), rstd.reshape(-1)]).float()
    dx, dgamma, dbeta = ln.backward(x.to(dtype), gamma, stats, dy.to(dtype), out=out, workspace=workspace)
    axis, other = (1, (0, 2)) if first else (2, (0, 1))
    mean, rstd = mean.unsqueeze(axis), rstd.unsqueeze(axis)
    xhat = (x - mean) * rstd
    assert torch.equal(dgamma, (dy * xhat).sum(other).to(torch.float32).to(dtype))
    assert torch.equal(dbeta, dy.sum(other).to(torch.float32).to(dtype))
    gd = dy * gamma.double().view([1, -1, 1] if first else [1, 1, -1])
    c1, c2 = gd.mean(axis, keepdim=True), (gd * xhat).mean(axis, keepdim=True)
    want = rstd * (gd - c1 - xhat * c2)
    tol = K * U * (gd.abs().mean(axis, keepdim=True) + xhat.abs() * (gd * xhat).abs().mean(axis, keepdim=True))
    tol = HALF[dtype] * want.abs() + rstd * (tol + 8 * U * (gd.abs() + c1.abs() + (xhat * c2).abs()))
    assert ((dx.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("tokens", [0, 1])
def test_more_channels_than_one_dimension_of_a_grid_has_columns(tokens):
    """2^26 + 5 channels: dgamma and dbeta are 2^27 + 10 columns, more than 2^32 threads. With one token they are dy xhat
    and dy: a few roundings and the storage type's; with none 0."""
    C = (1 << 26) + 5
    g = torch.Generator(device=DEV).manual_seed(22)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV).to(B)
    x, dy, gamma = rand(1, C, tokens), rand(1, C, tokens), rand(C)
    x.mul_(2.0), dy.add_(1.0)
    ln = LayerNorm.for_tensor(x, "channels_first")
    nan = lambda *s: torch.full(s, float("nan"), dtype=B, device=DEV)
    out = (nan(1, C, tokens), nan(C), nan(C))
    stats = torch.tensor([[0.25], [0.5]], device=DEV)[:, :tokens].contiguous()
    dx, dgamma, dbeta = ln.backward(x, gamma, stats, dy, out=out)
    torch.cuda.synchronize()
    if tokens == 0:
        assert not dgamma.any() and not dbeta.any()
        return
    xhat, d = ((x.double() - 0.25) * 0.5).view(-1), dy.double().view(-1)
    want = d * xhat
    assert ((dgamma.double() - want).abs() <= (HALF[B] + 8 * U) * want.abs()).all()
    assert torch.equal(dbeta, dy.view(-1))
    gd = d * gamma.double()
    c1, c2 = gd.mean(), (gd * xhat).mean()
    want = 0.5 * (gd - c1 - xhat * c2)
    # 2^18 terms a thread of the means, then the lanes' and waves'
    k = (C // 256 + 30) * U
    tol = HALF[B] * want.abs() + 0.5 * (k * (gd.abs().mean() + xhat.abs() * (gd * xhat).abs().mean())
                                        + 8 * U * (gd.abs() + c1.abs() + (xhat * c2).abs()))
    assert ((dx.double().view(-1) - want).abs() <= tol).all()
