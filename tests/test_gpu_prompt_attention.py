"""Attention over whole prompts on the GPU, forward and backward, against its definition in 64 bits (the bounds are derived
in attention_reference)."""
import numpy as np
import pytest
import torch

import attention_reference as ref
from ff_input_projection_amd import (EALIAS, EALIGN, EINVAL, FusedProjection, FusedProjError, KVCache, LayerNorm,
                                     PromptAttention, Rope)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


class Case:
    def __init__(self, batch, tokens, heads, kvh, hd, causal=True, sequences=0, extents=None, layout="heads", seed=0, scale=0.0):
        self.b, self.t, self.h, self.kvh, self.hd = batch, tokens, heads, kvh, hd
        self.causal, self.sequences, self.scale = causal, sequences, scale or hd ** -0.5
        self.extents = extents
        rng = np.random.default_rng(seed)
        make = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(BF16)
        self.q, self.k, self.v, self.do = make(batch, heads, tokens, hd), make(batch, kvh, tokens, hd), make(batch, kvh, tokens, hd), make(batch, tokens, heads, hd)
        self.layout = layout
        self.where = ref.spans(batch, tokens, sequences, extents)

    def on_gpu(self):
        """q, k, v as the layout has them, d_o, extents."""
        q, k, v = (x.to(DEV) for x in (self.q, self.k, self.v))
        if self.layout == "heads":
            q, k, v = (x.reshape(-1, self.t, self.hd) for x in (q, k, v))
        else:                                           # side by side in rows of a wider tensor
            rows = torch.cat([x.transpose(1, 2).reshape(self.b, self.t, -1) for x in (q, k, v, k[..., :8])], -1)
            q, k, v = (x.view(self.b, self.t, -1, self.hd).transpose(1, 2)
                       for x in rows.split([self.h * self.hd, self.kvh * self.hd, self.kvh * self.hd, self.kvh * 8], -1)[:3])
        e = None if self.extents is None else torch.tensor(self.extents, dtype=torch.int32, device=DEV)
        return q, k, v, self.do.to(DEV).view(self.b, self.t, -1), e

    def plan(self, q, k, v):
        return PromptAttention.for_tensors(q, k, v, batch=self.b, causal=self.causal, sequences=self.sequences,
                                           sm_scale=0.0 if self.scale == self.hd ** -0.5 else self.scale)

    def run(self):
        """Into outputs and a workspace full of NaN."""
        q, k, v, do, e = self.on_gpu()
        plan = self.plan(q, k, v)
        nan = lambda s, dtype=BF16: torch.full(s, float("nan"), dtype=dtype, device=DEV)
        ws = torch.full((plan.workspace_bytes() // 4 + 4,), float("nan"), device=DEV)
        o, lse = plan(q, k, v, e, out=(nan((self.b, self.t, self.h * self.hd)), nan((self.b * self.h, self.t), torch.float32)))
        grads = plan.backward(q, k, v, o, lse, do, e, out=tuple(nan(x.shape) for x in (q, k, v)), workspace=ws)
        torch.cuda.synchronize()
        got = {"o": o.view(self.b, self.t, self.h, self.hd), "lse": lse.view(self.b, self.h, self.t)}
        for name, x, like in zip(("dq", "dk", "dv"), grads, (self.q, self.k, self.v)):
            got[name] = x.view(like.shape)
        return {name: x.double().cpu().numpy() for name, x in got.items()}

    def want(self):
        return ref.attention(*(x.double().numpy() for x in (self.q, self.k, self.v)), self.causal, self.scale, self.where,
                             self.do.double().numpy())


def check(got, want):
    for name, (value, bound) in want.items():
        x = got[name]
        none = ~np.isfinite(value)                       # lse of tokens of no sequence
        assert np.array_equal(x[none], value[none]), name
        err = np.abs(x[~none] - value[~none])
        print(f"[attention] {name} max err/tol {(err / np.maximum(bound[~none], 1e-300)).max(initial=0.0):.3g}", flush=True)
        assert (err <= bound[~none]).all(), name


CASES = [dict(batch=1, tokens=1, heads=1, kvh=1, hd=8), dict(batch=2, tokens=2, heads=2, kvh=1, hd=16, causal=False)]
CASES += [dict(batch=1, tokens=t, heads=2, kvh=1, hd=64, causal=c) for t in (31, 32, 33, 64, 65, 127, 128, 129, 200, 321) for c in (True, False)]
CASES += [dict(batch=1, tokens=150, heads=3, kvh=1, hd=hd, causal=c) for hd in (8, 24, 32, 40, 72, 80, 96, 104, 128, 136, 192, 200, 256) for c in (True, False)]
CASES += [
    # padded batches: lengths of nothing, of one, past the padding, below 0
    dict(batch=5, tokens=140, heads=4, kvh=2, hd=64, extents=[0, 1, 140, 999, -3]),
    dict(batch=4, tokens=140, heads=4, kvh=4, hd=128, causal=False, extents=[0, 1, 97, 140]),
    dict(batch=3, tokens=70, heads=4, kvh=1, hd=80, causal=False, extents=[33, 64, 65], layout="qkv"),
    # packed: empty sequences, tokens before the first and behind the last, many short ones, borders at tiles' ends
    dict(batch=1, tokens=300, heads=4, kvh=2, hd=64, sequences=6, extents=[5, 5, 70, 128, 128, 256, 290]),
    dict(batch=1, tokens=300, heads=4, kvh=2, hd=128, sequences=3, extents=[0, 131, 132, 300], causal=False),
    dict(batch=1, tokens=257, heads=2, kvh=1, hd=96, sequences=40, extents=[6 * i for i in range(41)]),
    dict(batch=1, tokens=130, heads=2, kvh=2, hd=32, sequences=130, extents=list(range(131)), causal=False),
    dict(batch=1, tokens=260, heads=2, kvh=1, hd=192, sequences=2, extents=[0, 129, 260], layout="qkv"),
    dict(batch=1, tokens=200, heads=2, kvh=1, hd=64, sequences=300, extents=[0] * 150 + [77] * 100 + [200] * 51),
    dict(batch=1, tokens=200, heads=2, kvh=1, hd=64, sequences=2, extents=[0, 0, 0]),
    dict(batch=1, tokens=200, heads=2, kvh=1, hd=64, sequences=2, extents=[200, 200, 200]),
    dict(batch=1, tokens=200, heads=2, kvh=1, hd=64, sequences=2, extents=[-7, 90, 2 ** 31 - 1]),
    # offsets that do not ascend
    dict(batch=1, tokens=200, heads=2, kvh=1, hd=64, sequences=4, extents=[20, 150, 60, 250, 180]),
    dict(batch=1, tokens=200, heads=2, kvh=1, hd=64, sequences=2, extents=[150, 60, 20]),
    # groups
    dict(batch=2, tokens=90, heads=12, kvh=1, hd=32), dict(batch=2, tokens=131, heads=6, kvh=3, hd=128, layout="qkv"),
    dict(batch=1, tokens=700, heads=4, kvh=1, hd=64), dict(batch=1, tokens=1100, heads=2, kvh=2, hd=128, causal=False),
    # many heads: workgroups of other shapes than the small calls above have
    *(dict(batch=2, tokens=131, heads=128, kvh=128, hd=hd, causal=c) for hd, c in ((32, True), (64, False), (64, True), (80, True), (96, False), (128, True), (104, False))),
    *(dict(batch=2, tokens=150, heads=128, kvh=64, hd=hd, causal=c, extents=[150, 97]) for hd, c in ((16, True), (64, False), (72, True), (128, False), (120, True))),
    dict(batch=1, tokens=515, heads=128, kvh=128, hd=64, sequences=5, extents=[2, 60, 260, 261, 400, 513]),
    dict(batch=1, tokens=515, heads=128, kvh=64, hd=128, sequences=5, extents=[2, 60, 260, 261, 400, 513], causal=False),
    # a group's heads in parts (few keys), also of an odd number of heads
    dict(batch=1, tokens=300, heads=15, kvh=3, hd=64, sequences=2, extents=[3, 130, 290]), dict(batch=1, tokens=260, heads=8, kvh=1, hd=128, causal=False),
    dict(batch=1, tokens=300, heads=6, kvh=2, hd=200), dict(batch=2, tokens=257, heads=5, kvh=1, hd=256, extents=[257, 100], layout="qkv"),
    # steep and flat
    dict(batch=1, tokens=150, heads=2, kvh=2, hd=64, scale=3.0), dict(batch=1, tokens=150, heads=2, kvh=2, hd=64, scale=1e-6),
]


@pytest.mark.parametrize("kw", CASES, ids=["_".join(str(x) if not isinstance(x, list) else f"e{sum(x) % 1000}" for x in c.values()) for c in CASES])
def test_forward_and_backward(kw):
    print(f"[case] attention {kw}", flush=True)
    c = Case(**kw)
    check(c.run(), c.want())


def test_maxima_that_move():
    """Logits that rise, and fall, by hundreds along the keys, by steps below and above what the maximum waits for."""
    for slope in (0.5, 6.0, -6.0):
        c = Case(1, 300, 2, 1, 64, causal=False)
        up = torch.linspace(0, 1, 300)[None, None, :, None] * slope
        c.q, c.k = (c.q.float() * 0.5 + 2.0).to(BF16), (c.k.float() * 0.3 + up).to(BF16)
        check(c.run(), c.want())


@pytest.mark.parametrize("kw", [dict(batch=1, tokens=150, heads=2, kvh=1, hd=64), dict(batch=1, tokens=150, heads=2, kvh=1, hd=80, causal=False),
                                dict(batch=1, tokens=170, heads=2, kvh=1, hd=128, sequences=4, extents=[3, 40, 90, 90, 160]),
                                dict(batch=2, tokens=140, heads=1, kvh=1, hd=64, extents=[100, 37]),
                                dict(batch=1, tokens=150, heads=2, kvh=2, hd=256, sequences=2, extents=[0, 77, 150], causal=False),
                                dict(batch=1, tokens=150, heads=256, kvh=128, hd=128, extents=[133]),
                                dict(batch=1, tokens=150, heads=256, kvh=256, hd=64, sequences=2, extents=[0, 77, 141])])
@pytest.mark.parametrize("which", ["v", "k", "q", "do"])
def test_what_is_not_finite_reaches_those_that_see_it(kw, which):
    print(f"[case] attention {which} {kw}", flush=True)
    c = Case(**kw)
    x = getattr(c, which) if which != "do" else c.do.transpose(1, 2)
    places = [(c.t // 3, 5, float("nan")), (c.t - 30, 2, float("nan")), (c.t // 2, 7, float("nan"))]
    if which == "v":
        places[1:] = [(c.t - 30, 2, float("inf")), (c.t // 2, 7, float("-inf"))]
    for s, d, value in places:
        x[0, -1, s, d] = value
    # what no token sees: rows of no sequence
    outside = np.ones((c.b, c.t), dtype=bool)
    for row, x0, x1 in c.where:
        outside[row, x0:x1] = False
    for y in (c.q, c.k, c.v, c.do.transpose(1, 2)):
        y.transpose(1, 2)[torch.from_numpy(outside)] = float("nan")
    got = c.run()
    want = ref.not_finite(*(y.double().numpy() for y in (c.q, c.k, c.v)), c.causal, c.scale, c.where, c.do.double().numpy())
    # the bounds of the finite values: with the places set to 0, which changes what sees them
    for name in ("o", "lse", "dq", "dk", "dv"):
        if which == "v" and name in ("dq", "dk"):
            # where v is infinite, D and dp are: NaN in the row's ds, as inf - inf
            assert np.array_equal(np.isfinite(got[name]), np.isfinite(want[name])), name
        else:
            assert np.array_equal(np.isnan(got[name]), np.isnan(want[name])), name
        fine = np.isfinite(want[name])
        assert np.array_equal(np.isinf(got[name]) & ~np.isnan(want[name]), np.isinf(want[name])) or (which == "v" and name in ("dq", "dk")), name
        big = np.abs(want[name][fine]).max(initial=1.0)
        assert np.abs(got[name][fine] - want[name][fine]).max(initial=0.0) <= 2.0 ** -4 * big, name


def test_results_do_not_depend_on_timing():
    c = Case(2, 500, 8, 2, 64, extents=[500, 333])
    first = c.run()
    for _ in range(3):
        again = c.run()
        assert all(np.array_equal(first[n], again[n]) for n in first)


def test_heads_that_share_memory():
    """k and v of stride 0: one k/v head that all heads read, as an expanded view; its gradients come a head each."""
    c = Case(1, 100, 4, 4, 64)
    q, k, v, do, _ = c.on_gpu()
    q, k, v = q[None], k[None, :1].expand(-1, 4, -1, -1), v[None, :1].expand(-1, 4, -1, -1)
    c.k, c.v = c.k[:, :1].expand(-1, 4, -1, -1).clone(), c.v[:, :1].expand(-1, 4, -1, -1).clone()
    plan = PromptAttention.for_tensors(q, k, v)
    o, lse = plan(q, k, v)
    grads = plan.backward(q, k, v, o, lse, do)
    got = {"o": o.view(1, 100, 4, 64), "lse": lse[None], **dict(zip(("dq", "dk", "dv"), grads))}
    check({n: x.double().cpu().numpy() for n, x in got.items()}, c.want())


def test_captured_with_extents_that_change():
    c = Case(1, 300, 4, 2, 64, sequences=3, extents=[0, 100, 200, 300])
    q, k, v, do, e = c.on_gpu()
    plan = c.plan(q, k, v)

    def step():
        o, lse = plan(q, k, v, e)
        return o, lse, *plan.backward(q, k, v, o, lse, do, e)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for cuts in ([0, 100, 200, 300], [0, 7, 150, 280], [40, 40, 41, 300], [0, 0, 0, 0]):
        e.copy_(torch.tensor(cuts, dtype=torch.int32))
        q.copy_(torch.randn(q.shape, device=DEV).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_on_other_streams_at_once():
    c = Case(2, 400, 8, 4, 64, extents=[400, 130])
    q, k, v, do, e = c.on_gpu()
    plan = c.plan(q, k, v)
    o, lse = plan(q, k, v, e)
    want = (o, lse, *plan.backward(q, k, v, o, lse, do, e))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for st in streams:
        o, lse = plan(q, k, v, e, stream=st)
        got.append((o, lse, *plan.backward(q, k, v, o, lse, do, e, stream=st)))
    for st in streams:
        st.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_without_lse_and_empty():
    c = Case(1, 90, 2, 2, 64)
    q, k, v, do, _ = c.on_gpu()
    plan = c.plan(q, k, v)
    want = plan(q, k, v)[0]
    out = torch.empty_like(want)
    assert plan(q, k, v, out=(out, None))[1] is None
    assert torch.equal(out, want)
    none = PromptAttention(0, 5, 4, 64)
    x = torch.empty((0, 5, 64), dtype=BF16, device=DEV)
    o, lse = none(x, x, x)
    assert o.shape == (0, 5, 256) and lse.shape == (0, 5)
    assert none.backward(x, x, x, o, lse, o)[0].shape == (0, 5, 64)


def test_far_rows():
    """Tokens more than 4 GiB from their tensor's start: the last sequence of a wide one, against the same rows alone."""
    width, tokens = 1 << 15, (1 << 16) + 1024
    big = torch.zeros((1, tokens, width), dtype=BF16, device=DEV)
    assert big.numel() * 2 > 1 << 32
    n = 200
    g = torch.Generator(device=DEV).manual_seed(1)
    big[0, -n:, -3 * 64:] = torch.randn((n, 3 * 64), generator=g, device=DEV).to(BF16)
    q, k, v = (big[:, :, width - (3 - i) * 64:width - (2 - i) * 64].unsqueeze(1) for i in range(3))
    e = torch.tensor([tokens - n, tokens], dtype=torch.int32, device=DEV)
    plan = PromptAttention.for_tensors(q, k, v, sequences=1)
    do = torch.randn((1, tokens, 64), generator=g, device=DEV).to(BF16)
    o, lse = plan(q, k, v, e)
    grads = plan.backward(q, k, v, o, lse, do, e)
    qs, ks, vs = (x[:, :, -n:].contiguous() for x in (q, k, v))
    small = PromptAttention.for_tensors(qs, ks, vs)
    o2, lse2 = small(qs, ks, vs)
    # other tiles (the sequence begins inside one of 128 tokens), so other orders of the sums and roundings of p
    assert (o[0, -n:].float() - o2[0].float()).abs().max() <= 2.0 ** -6 * o2.float().abs().max()
    assert not o[0, :-n].any() and torch.isneginf(lse[0, :-n]).all()
    for a, b in zip(grads, small.backward(qs, ks, vs, o2, lse2, do[:, -n:].contiguous())):
        assert (a[0, 0, -n:].float() - b[0, 0].float()).abs().max() <= 2.0 ** -6 * b.float().abs().max()
        assert not a[0, 0, :-n].any()


def test_refusals():
    c = Case(1, 40, 4, 2, 64, sequences=2, extents=[0, 9, 40])
    q, k, v, do, e = c.on_gpu()
    plan = c.plan(q, k, v)
    o, lse = plan(q, k, v, e)
    dq, dk, dv = plan.backward(q, k, v, o, lse, do, e)
    ws = plan.alloc_workspace(DEV)
    lib, h, p = plan._lib, plan._h, lambda t: None if t is None else t.data_ptr()
    st = torch.cuda.current_stream().cuda_stream
    run = lambda q=q, k=k, v=v, e=e, o=o, lse=lse, more=0: lib.prompt_attention_run(h, p(q), p(k), p(v), p(e), p(o) + more if o is not None else None, p(lse), st)
    assert run(q=None) == EINVAL and run(e=None) == EINVAL and run(o=None) == EINVAL
    assert run(more=2) == EALIGN and run(k=k.flatten()[1:]) == EALIGN
    assert run(o=q) == EALIAS and run(o=v) == EALIAS and run(lse=o) == EALIAS and run(lse=e) == EALIAS
    back = lambda n=ws.numel(), o=o, dq=dq, dk=dk, dv=dv, ws=ws, lse=lse: lib.prompt_attention_backward(h, p(q), p(k), p(v), p(e), p(o), p(lse), p(do), p(dq), p(dk), p(dv), p(ws), n, st)
    assert back(n=ws.numel() - 1) == EINVAL and back(ws=None) == EINVAL and back(lse=None) == EINVAL and back(dv=None) == EINVAL
    assert back(ws=ws[4:]) == EALIGN
    assert back(dq=q) == EALIAS and back(dk=dv) == EALIAS and back(dq=o) == EALIAS and back(dv=ws) == EALIAS
    with pytest.raises(ValueError):
        plan(q, k, v)
    with pytest.raises(ValueError):
        plan(q, k, v, e[:2])
    with pytest.raises(ValueError):
        plan(q, k, v, e.long())
    with pytest.raises(ValueError):
        plan(q[None], k[None], v[None], e)
    with pytest.raises(ValueError):
        plan(q.float(), k, v, e)
    with pytest.raises(TypeError):
        plan(q.cpu(), k, v, e)
    with pytest.raises(ValueError):
        plan(q, k.cpu(), v, e)
    with pytest.raises(ValueError):
        plan.backward(q, k, v, o, lse, do[:, :8], e)
    with pytest.raises(ValueError):
        plan.backward(q, k, v, o, lse, do, e, out=(dq, dk, dk[:1]))
    with pytest.raises(FusedProjError):
        plan.backward(q, k, v, o, lse, do, e, workspace=ws[:64])
    plan.close()
    with pytest.raises(FusedProjError):
        plan(q, k, v, e)


@pytest.mark.parametrize("kw", [dict(batch=1, tokens=140, heads=4, kvh=2, hd=64), dict(batch=1, tokens=140, heads=2, kvh=1, hd=96, causal=False, sequences=2, extents=[0, 60, 133])])
def test_gradients_against_differences(kw):
    """The gradients along a direction, against a central difference of the reference's sum(do o): off by their bounds, and by
    the difference's own error (h^2 times a third derivative of order 1 a term, and roundings over h)."""
    c = Case(**kw)
    got, want = c.run(), c.want()
    rng = np.random.default_rng(9)
    x = {n: getattr(c, n).double().numpy() for n in ("q", "k", "v")}
    do = c.do.double().numpy()
    loss = lambda y: (ref.attention(y["q"], y["k"], y["v"], c.causal, c.scale, c.where)["o"][0] * do).sum()
    for n in ("q", "k", "v"):
        r = rng.standard_normal(x[n].shape)
        h = 1e-4
        diff = (loss({**x, n: x[n] + h * r}) - loss({**x, n: x[n] - h * r})) / (2 * h)
        slope = (got["d" + n] * r).sum()
        assert abs(diff - slope) <= (want["d" + n][1] * np.abs(r)).sum() + 1e-4


def test_a_block_in_training():
    """norm, projection, rotation by positions, attention, and all four backward passes: each gradient against a run of the
    same block in 64 bits (by autograd on the CPU). Bounds: the roundings to bf16 on the way - of the norm's output, qkv, q
    and k, p, o (5 forward), and of their gradients and ds (6 back), and of the result - each of half a step, add up to at
    most 12 half steps of a value if all point one way; they are independent, and what is compared is the 2-norm."""
    b, t, ch, h, kvh, hd = 1, 160, 128, 4, 2, 64
    g = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=g, dtype=torch.float64).to(BF16)
    x, w = rand(b, t, ch), (rand(ch, (h + 2 * kvh) * hd).double() / ch ** 0.5).to(BF16)
    gamma, beta, do = (1 + 0.1 * rand(ch).double()).to(BF16), (0.1 * rand(ch).double()).to(BF16), rand(b, t, h * hd)
    cuts = [0, 50, 51, 160]
    at = torch.cat([torch.arange(m - n) for n, m in zip(cuts, cuts[1:])]).to(torch.int32)[None]

    dx_, dw_, dgamma_, dbeta_ = (v.double().requires_grad_() for v in (x, w, gamma, beta))
    y = torch.nn.functional.layer_norm(dx_, (ch,), dgamma_, dbeta_, 1e-5)
    rows = (y @ dw_).view(b, t, -1, hd).transpose(1, 2)
    theta = torch.tensor([10000.0 ** (-2 * i / hd) for i in range(hd // 2)], dtype=torch.float64)
    phi = at.double()[:, None, :, None] * theta

    def turn(z):
        p, s = z[..., :hd // 2], z[..., hd // 2:]
        return torch.cat([p * phi.cos() - s * phi.sin(), s * phi.cos() + p * phi.sin()], -1)

    q, k, v = turn(rows[:, :h]), turn(rows[:, h:h + kvh]), rows[:, h + kvh:]
    k, v = (z.repeat_interleave(h // kvh, 1) for z in (k, v))
    of = torch.bucketize(torch.arange(t), torch.tensor(cuts), right=True)
    see = (of[:, None] == of) & (torch.arange(t) <= torch.arange(t)[:, None])
    p = (q @ k.transpose(-1, -2) * hd ** -0.5).masked_fill(~see, -np.inf).softmax(-1)
    o_ = (p @ v).transpose(1, 2).reshape(b, t, -1)
    o_.backward(do.double())

    xg, wg, gg, bg, dg = (z.to(DEV) for z in (x, w, gamma, beta, do))
    norm = LayerNorm.for_tensor(xg, "tokens_last")
    proj = FusedProjection.for_tensor(xg, "tokens_last", ff_dim=w.shape[1])
    rope = Rope(b, t, h, hd, n_kv_heads=kvh)
    attend = PromptAttention(b, t, h, hd, n_kv_heads=kvh, sequences=3)
    at, e = at.to(DEV), torch.tensor(cuts, dtype=torch.int32, device=DEV)
    y, stats = norm(xg, gg, bg)
    q, k, v = rope(proj(y, wg)[0], at)
    o, lse = attend(q, k, v, e)
    dqkv = rope.backward(*attend.backward(q, k, v, o, lse, dg, e), at)
    dy, dw, _ = proj.backward(y, wg, None, d_ff=dqkv)
    dx, dgamma, dbeta = norm.backward(xg, gg, stats, dy)
    for name, got, want in (("o", o, o_), ("dw", dw, dw_.grad), ("dx", dx, dx_.grad), ("dgamma", dgamma, dgamma_.grad), ("dbeta", dbeta, dbeta_.grad)):
        off = (got.double().cpu() - want.detach()).norm() / want.detach().norm()
        print(f"[block] {name} {off:.3g}", flush=True)
        assert off <= 12 * 2.0 ** -8, name


def test_a_prompt_then_single_tokens():
    """A prompt through this attention and its k and v into a cache in 8 bits; the next token's attention over the cache is
    this attention's of the whole, but for the cache's rounding (rows of 64 normal values, scale at most 8 / 255, each off by
    half a step, and the logits' shift by it)."""
    b, t, h, kvh, hd = 2, 130, 4, 2, 64
    c = Case(b, t, h, kvh, hd)
    q, k, v, _, _ = c.on_gpu()
    whole = PromptAttention.for_tensors(q, k, v, batch=b)(q, k, v)[0]
    kw = dict(n_kv_heads=kvh, bits=8, page_size=16, n_pages=2 * 9, max_pages=9)
    prompt, step = KVCache(b, t, h, hd, **kw), KVCache(b, 1, h, hd, **kw)
    storage = prompt.alloc_storage(DEV)
    table = torch.arange(18, dtype=torch.int32, device=DEV).view(2, 9)
    n = torch.full((b,), t, dtype=torch.int32, device=DEV)
    prompt.write(storage, k, v, table, n)
    last = step.attend(storage, q[:, -1:].contiguous(), table, n)
    assert (last[:, 0].float() - whole[:, -1].float()).abs().max() <= 0.05


SHORT = [dict(batch=7, tokens=t, heads=4, kvh=2, hd=hd, causal=c) for t, hd, c in
         ((1, 128, True), (2, 256, False), (17, 8, True), (17, 64, False), (31, 96, True), (32, 32, False), (32, 128, True), (29, 136, True),
          (32, 192, False), (30, 256, True))]
SHORT += [dict(batch=4, tokens=t, heads=128, kvh=64, hd=hd, causal=c) for t, hd, c in
          ((33, 64, True), (50, 32, False), (64, 128, True), (64, 64, False), (49, 80, True), (40, 96, False), (57, 104, True), (36, 192, True),
           (64, 200, False), (63, 256, True))]
SHORT += [
    dict(batch=5, tokens=30, heads=4, kvh=1, hd=64, extents=[0, 1, 30, 99, -2], causal=False),
    dict(batch=4, tokens=60, heads=128, kvh=128, hd=128, extents=[0, 33, 60, 7], layout="qkv"),
    dict(batch=1, tokens=31, heads=6, kvh=3, hd=128, sequences=5, extents=[2, 2, 9, 10, 25, 30]),
    dict(batch=1, tokens=61, heads=512, kvh=256, hd=64, sequences=4, extents=[1, 20, 20, 47, 60], causal=False),
]


@pytest.mark.parametrize("kw", SHORT, ids=["_".join(str(x) if not isinstance(x, list) else f"e{sum(x) % 1000}" for x in c.values()) for c in SHORT])
def test_short_sequences(kw):
    print(f"[case] attention {kw}", flush=True)
    c = Case(**kw)
    check(c.run(), c.want())


@pytest.mark.parametrize("kw", [dict(batch=1, tokens=64, heads=512, kvh=256, hd=128, extents=[61]), dict(batch=3, tokens=32, heads=2, kvh=1, hd=64),
                                dict(batch=1, tokens=60, heads=512, kvh=512, hd=64, sequences=2, extents=[0, 32, 58], causal=False)])
@pytest.mark.parametrize("which", ["v", "k", "q", "do"])
def test_short_sequences_that_are_not_finite(kw, which):
    test_what_is_not_finite_reaches_those_that_see_it(kw, which)
