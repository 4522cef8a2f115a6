"""Rotary positions on the GPU against their definition in 64 bits (the bound is derived in rope_reference.rotate)."""
import numpy as np
import pytest
import torch

import rope_reference as ref
from ff_input_projection_amd import EALIAS, EALIGN, EINVAL, FusedProjection, FusedProjError, Rope, SplitRope

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF16, F32 = torch.bfloat16, torch.float32
SCALED = dict(scaling="by_parts", factor=8.0, original_tokens=512, low_turns=1.0, high_turns=20.0, magnitude=1.2)


class Case:
    def __init__(self, dtype, batch, tokens, heads, kvh, hd, dims, pairs, order="contiguous", seed=0, positions="far", **kw):
        self.dtype, self.b, self.t, self.h, self.kvh, self.hd, self.pairs, self.order = dtype, batch, tokens, heads, kvh, hd, pairs, order
        self.magnitude = kw.get("magnitude", 1.0) or 1.0
        rng = np.random.default_rng(seed)
        self.theta = ref.frequencies(dims or hd, **{("base" if k == "rope_base" else k): v for k, v in kw.items() if k != "magnitude"})
        self.plan = Rope(batch, tokens, heads, hd, n_kv_heads=kvh, qkv_order=order, rope_dims=dims, pairs=pairs, dtype=dtype, **kw)
        shapes = [(batch, n, tokens, hd) for n in (heads, kvh, kvh)]
        self.x = [torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dtype) for s in shapes]
        self.at = {"far": lambda: rng.integers(-2 ** 31, 2 ** 31, (batch, tokens)), "none": lambda: np.tile(np.arange(tokens), (batch, 1)),
                   "near": lambda: rng.integers(0, 8192, (batch, 1)) + np.arange(tokens)}[positions]()
        self.positions = None if positions == "none" else torch.from_numpy(self.at.astype(np.int32)).to(DEV)

    def on_gpu(self):
        return [x.view(-1, self.t, self.hd).to(DEV) for x in self.x]

    def rows(self):
        x = ref.join(*(x.double().numpy() for x in self.x), self.order)
        return torch.from_numpy(np.ascontiguousarray(x)).to(self.dtype).view(self.b, self.t, -1).to(DEV)

    def want(self, back):
        """[(y, tolerance)] of q and k; v is copied."""
        return [ref.rotate(x.double().numpy(), self.at, self.theta, self.pairs, self.magnitude, back, EPS[self.dtype]) for x in self.x[:2]]


def within(got, want, tol):
    got = got.double().cpu().numpy().reshape(want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    err = np.abs(got[fine] - want[fine])
    print(f"[rope] max err/tol {(err / np.maximum(tol[fine], 1e-300)).max(initial=0.0):.3g}", flush=True)
    assert (err <= tol[fine]).all()


CASES = [  # dtype, batch, tokens, heads, kvh, hd, dims, pairs, order
    (BF16, 1, 1, 1, 1, 8, 0, "half"), (BF16, 1, 1, 1, 1, 8, 2, "interleaved"), (F32, 1, 1, 1, 1, 8, 0, "half"),
    (BF16, 16, 1, 32, 8, 128, 0, "half"), (BF16, 2, 37, 6, 2, 64, 0, "half", "grouped"), (BF16, 2, 37, 6, 2, 64, 0, "interleaved", "grouped"),
    (BF16, 3, 50, 16, 4, 32, 8, "half", "grouped"), (F32, 3, 50, 16, 4, 32, 8, "half", "grouped"), (BF16, 2, 19, 5, 5, 80, 20, "half"),
    (BF16, 2, 19, 5, 5, 80, 22, "half"), (F32, 2, 19, 5, 5, 80, 22, "half"), (F32, 2, 19, 5, 1, 80, 20, "interleaved"),
    (BF16, 1, 130, 3, 1, 96, 50, "interleaved"), (F32, 2, 33, 7, 7, 256, 0, "half"), (BF16, 1, 9, 2, 1, 4096, 0, "half"),
    (F32, 1, 9, 2, 1, 24, 22, "interleaved"), (BF16, 1, 700, 4, 2, 40, 24, "half"), (F32, 5, 3, 2, 2, 72, 36, "half", "grouped"),
]


@pytest.mark.parametrize("case", CASES, ids=["_".join(str(x).replace("torch.", "") for x in c) for c in CASES])
def test_forward_and_backward(case):
    print(f"[case] rope {case}", flush=True)
    c = Case(*case)
    q, k, v = c.plan(c.rows(), c.positions)
    dqkv = c.plan.backward(*c.on_gpu(), c.positions)
    rq, rk = c.plan.rotate(*c.on_gpu()[:2], c.positions)
    gq, gk = c.plan.rotate_backward(*c.on_gpu()[:2], c.positions)
    torch.cuda.synchronize()
    for got, again, (want, tol) in zip((q, k), (rq, rk), c.want(False)):
        within(got, want, tol)
        assert torch.equal(got, again)
    assert torch.equal(v.cpu().view(c.x[2].shape), c.x[2])
    parts = ref.split(dqkv.double().cpu().numpy().reshape(c.b, c.t, -1, c.hd), c.h, c.kvh, c.order)
    for got, again, (want, tol) in zip(parts, (gq, gk), c.want(True)):
        within(torch.from_numpy(np.ascontiguousarray(got)), want, tol)
        assert np.array_equal(got, again.double().cpu().numpy().reshape(got.shape))
    assert np.array_equal(parts[2], c.x[2].double().numpy())


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=4.0), SCALED, dict(rope_base=5e5), dict(rope_base=0.5),
                                dict(magnitude=-0.25), dict(magnitude=0.0),
                                dict(scaling="by_parts", factor=0.15, original_tokens=1)])
@pytest.mark.parametrize("dtype,pairs,positions", [(BF16, "half", "near"), (F32, "interleaved", "none"), (F32, "half", "far")])
def test_frequencies_and_positions(dtype, pairs, positions, kw):
    print(f"[case] rope {dtype} {pairs} {positions} {kw}", flush=True)
    c = Case(dtype, 2, 65, 4, 2, 64, 48, pairs, positions=positions, **kw)
    for got, (want, tol) in zip(c.plan(c.rows(), c.positions)[:2], c.want(False)):
        within(got, want, tol)


def test_the_backward_pass_is_the_gradient():
    """The dot product of an upstream gradient with the difference of two outputs is that of the gradient with the
    difference of the inputs (the operator is linear); fp32, so both sums are off by U (n + 6) of their terms at most."""
    c, d = (Case(F32, 2, 31, 6, 2, 48, 32, "half", "grouped", seed=s, **SCALED) for s in (1, 2))
    dq, dk, dv = d.on_gpu()
    x1, x2 = c.rows(), d.rows()
    y = [(a.double() - b.double()) for a, b in zip(c.plan(x1, c.positions), c.plan(x2, c.positions))]
    g = c.plan.backward(dq, dk, dv, c.positions)
    left = sum((a * b.double()).sum() for a, b in zip(y, (dq, dk, dv)))
    right = (g.double() * (x1.double() - x2.double())).sum()
    size = sum((a.abs() * b.double().abs()).sum() for a, b in zip(y, (dq, dk, dv)))
    assert abs(left - right) <= 24 * 2.0 ** -24 * 2 * size


def test_in_place_and_outputs_given():
    c = Case(BF16, 3, 21, 6, 3, 64, 40, "half")
    q, k, v = c.on_gpu()
    want = c.plan.rotate(q, k, c.positions)
    out = (q.clone(), k.clone())
    assert c.plan.rotate(*out, c.positions, out=out)[0] is out[0]
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    c.plan.rotate_backward(*out, c.positions, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, c.plan.rotate_backward(*want, c.positions)))
    rows = c.rows()
    given = [torch.full_like(x, float("nan")) for x in (q, k, v)]
    c.plan(rows, c.positions, out=given)
    assert all(torch.equal(a, b) for a, b in zip(given, c.plan(rows, c.positions)))
    g = torch.full_like(rows, float("nan"))
    assert c.plan.backward(q, k, v, c.positions, out=g) is g
    assert torch.equal(g, c.plan.backward(q, k, v, c.positions))


def test_agrees_with_the_split_from_one_position():
    """A plan of SplitRope at an offset, whose angles are fp64 rounded to fp32 tables: each is off by the definition's bound."""
    c = Case(BF16, 2, 40, 8, 2, 64, 32, "half", "grouped", positions="none")
    rows = c.rows()
    old = SplitRope(2, 40, 8, 64, n_kv_heads=2, qkv_order="grouped", rope_dims=32, pos_offset=1000)(rows)
    c.at = c.at + 1000
    new = c.plan(rows, torch.from_numpy(c.at.astype(np.int32)).to(DEV))
    for a, b, (want, tol) in zip(old, new, c.want(False)):
        within(a, want, tol)
        within(b, want, tol)
    assert torch.equal(old[2], new[2])


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_what_is_not_finite_stays_in_its_pair(dtype, pairs):
    c = Case(dtype, 1, 12, 2, 2, 32, 24, pairs, positions="near")
    c.x[0][0, 0, 3, 1] = float("nan")
    c.x[0][0, 1, 5, 9] = float("inf")
    c.x[1][0, 1, 0, 30] = float("-inf")                     # copied
    for back in (False, True):
        if back:
            got = c.plan.rotate_backward(*c.on_gpu()[:2], c.positions)
        else:
            got = c.plan.rotate(*c.on_gpu()[:2], c.positions)
        for y, (want, tol) in zip(got, c.want(back)):
            within(y, want, tol)
        other = 13 if pairs == "half" else 0
        assert torch.isnan(got[0][0, 3]).nonzero().flatten().tolist() == sorted((1, other))
        assert got[1][1, 0, 30].item() == float("-inf")


def test_captured_with_positions_that_change():
    c = Case(BF16, 4, 1, 8, 2, 64, 0, "half", positions="near")
    rows = c.rows()
    c.plan(rows, c.positions)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c.plan(rows, c.positions)
    for step in range(3):
        c.positions += 1 + step
        rows.copy_(torch.randn(rows.shape, device=DEV).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, c.plan(rows, c.positions)))


def test_on_another_stream():
    c = Case(F32, 2, 64, 4, 4, 64, 0, "half")
    rows, want = c.rows(), c.plan(c.rows(), c.positions)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = c.plan(rows, c.positions, stream=st)
    back = c.plan.backward(*got, c.positions, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(back, c.plan.backward(*want, c.positions))


def test_an_empty_batch():
    plan = Rope(0, 5, 4, 64)
    q, k, v = plan(torch.empty((0, 5, 12 * 64), dtype=BF16, device=DEV))
    assert q.shape == (0, 5, 64) and k.shape == v.shape == (0, 5, 64)


def test_more_elements_than_31_bits():
    """Heads behind 2^31 elements of qkv: the last token's rows."""
    t, h, hd = 4096, 96, 256
    plan = Rope(8, t, h, hd, pairs="interleaved")
    rows = torch.zeros((8, t, 3 * h * hd), dtype=BF16, device=DEV)
    assert rows.numel() > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(3)
    rows[-1, -1] = torch.randn(rows.shape[-1], generator=g, device=DEV).to(BF16)
    small = Rope(1, 1, h, hd, pairs="interleaved")
    at = torch.full((1, 1), t - 1, dtype=torch.int32, device=DEV)
    want = small(rows[-1:, -1:].contiguous(), at)
    got = plan(rows)
    for a, b in zip(got, want):
        assert torch.equal(a.view(8, h, t, hd)[-1, :, -1], b[:, 0])
    back = plan.backward(*got)
    assert torch.equal(back[-1, -1], small.backward(*want, at)[0, 0])
    assert not back[0, 0].any()


def test_refusals():
    c = Case(BF16, 2, 8, 4, 2, 64, 0, "half")
    q, k, v = c.on_gpu()
    rows = c.rows()
    lib, h = c.plan._lib, c.plan._h
    p = lambda t: t.data_ptr()
    st = torch.cuda.current_stream().cuda_stream
    assert lib.rope_split(h, None, None, p(q), p(k), p(v), st) == EINVAL
    assert lib.rope_split(h, p(rows), None, p(q), None, p(v), st) == EINVAL
    assert lib.rope_split(h, p(rows) + 2, None, p(q), p(k), p(v), st) == EALIGN
    assert lib.rope_split(h, p(rows), p(c.positions) + 2, p(q), p(k), p(v), st) == EALIGN
    assert lib.rope_split(h, p(rows), None, p(q), p(k), p(k), st) == EALIAS
    assert lib.rope_split(h, p(rows), None, p(rows), p(k), p(v), st) == EALIAS
    assert lib.rope_split(h, p(rows), p(q), p(q), p(k), p(v), st) == EALIAS
    assert lib.rope_rotate(h, p(q), p(k), None, p(k), p(q), st) == EALIAS
    assert lib.rope_rotate(h, p(q), p(k), None, p(q) + 16, p(k), st) == EALIAS
    with pytest.raises(ValueError):
        c.plan(rows.float(), c.positions)
    with pytest.raises(ValueError):
        c.plan(rows[:, :4].contiguous(), c.positions)
    with pytest.raises(ValueError):
        c.plan(rows, c.positions.long())
    with pytest.raises(ValueError):
        c.plan(rows, c.positions[:1])
    with pytest.raises(ValueError):
        c.plan.rotate(q, k.transpose(0, 1), c.positions)
    with pytest.raises(TypeError):
        c.plan(rows.cpu(), c.positions)
    with pytest.raises(ValueError):
        c.plan(rows, c.positions.cpu())
    with pytest.raises(ValueError):
        c.plan(rows, c.positions, out=(q, k, v[:1]))
    c.plan.close()
    with pytest.raises(FusedProjError):
        c.plan(rows, c.positions)


def test_a_projection_in_training():
    """qkv of a projection without heads, split and rotated, and back: dx and dW are those of the projection that splits
    and rotates itself, up to the roundings of qkv and dqkv to bf16 that lie between."""
    b, t, ch, h, kvh, hd = 2, 48, 128, 4, 2, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn((b, t, ch), generator=g, device=DEV).to(BF16)
    w = (torch.randn((ch, (h + 2 * kvh) * hd), generator=g, device=DEV) / ch ** 0.5).to(BF16)
    plain = FusedProjection.for_tensor(x, "tokens_last", ff_dim=w.shape[1])
    whole = FusedProjection.for_tensor(x, "tokens_last", n_heads=h, head_dim=hd, n_kv_heads=kvh, rope=True)
    rope = Rope(b, t, h, hd, n_kv_heads=kvh)
    parts = rope(plain(x, w)[0])
    want = whole(x, w)[1:]
    for a, c in zip(parts, want):
        # one rounding of qkv more, of both elements of a pair
        tol = 2.0 ** -7 * c.float().abs() + 2.0 ** -8 * 1.5 * c.float().abs().amax(-1, keepdim=True)
        assert ((a.float() - c.float()).abs() <= tol).all()
    ups = [torch.randn(p.shape, generator=g, device=DEV).to(BF16) for p in parts]
    got = plain.backward(x, w, None, d_ff=rope.backward(*ups))
    ref_grads = whole.backward(x, w, None, dq=ups[0], dk=ups[1], dv=ups[2])
    for a, c in zip(got[:2], ref_grads[:2]):
        assert (a.float() - c.float()).norm() <= 2.0 ** -7 * c.float().norm()
