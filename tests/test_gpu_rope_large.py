"""Rotary positions in calls that are large enough for threads of four heads (rope.hip, kHeads): every type, pairing, width of
access and order, numbers of heads that four does not divide, in place, and what is not finite."""
import pytest
import torch

from test_gpu_rope import BF16, F32, SCALED, Case, test_forward_and_backward as forward_and_backward, within

pytestmark = pytest.mark.gpu

CASES = [  # dtype, batch, tokens, heads, kvh, hd, dims, pairs, order
    (BF16, 2, 5500, 9, 3, 64, 0, "half", "grouped"), (BF16, 1, 5500, 9, 3, 64, 0, "interleaved", "grouped"),
    (F32, 2, 2750, 9, 3, 64, 0, "half"), (F32, 1, 2750, 10, 5, 64, 36, "interleaved"), (BF16, 3, 450, 5, 5, 80, 20, "half"),
    (BF16, 1, 700, 5, 5, 80, 22, "half"), (F32, 1, 700, 7, 7, 80, 22, "half"), (BF16, 1, 5000, 13, 1, 32, 8, "half", "grouped"),
    (F32, 2, 1500, 6, 2, 72, 36, "half", "grouped"), (BF16, 1, 3700, 11, 1, 96, 50, "interleaved"),
]


def blocks_of_four(dtype, batch, tokens, heads, kvh, hd, dims, pairs, order="contiguous"):
    """Workgroups of the split, and of the rotation of q and k, with four heads a thread."""
    width, half = 16 // dtype.itemsize, (dims or hd) // 2
    if pairs == "half":
        while half % width:
            width //= 2
    items = batch * tokens * (hd - (half if pairs == "half" else 0)) // width
    return [(items + 255) // 256 * ((n + 3) // 4) for n in (heads + 2 * kvh, heads + kvh)]


@pytest.mark.parametrize("case", CASES, ids=["_".join(str(x).replace("torch.", "") for x in c) for c in CASES])
def test_threads_of_four_heads(case):
    assert min(blocks_of_four(*case)) >= 512
    forward_and_backward(case)


def test_both_ways_agree():
    """The same rows in a call of four heads a thread and in calls of one."""
    case = CASES[4]
    c = Case(*case)
    small = Case(case[0], 1, 50, *case[3:])
    assert max(blocks_of_four(case[0], 1, 50, *case[3:])) < 512
    rows = c.rows()
    whole = c.plan(rows, c.positions)
    for t in range(0, c.t, 50):
        part = small.plan(rows[1:2, t:t + 50].contiguous(), c.positions[1:2, t:t + 50].contiguous())
        for a, b in zip(whole, part):
            assert torch.equal(a.view(c.b, -1, c.t, c.hd)[1, :, t:t + 50], b)


@pytest.mark.parametrize("case", [CASES[0], CASES[3], CASES[5]], ids=["halves", "neighbours", "odd"])
def test_in_place(case):
    c = Case(*case, **SCALED)
    q, k, _ = c.on_gpu()
    want, back = c.plan.rotate(q, k, c.positions), c.plan.rotate_backward(q, k, c.positions)
    for got, (value, tol) in zip(want, c.want(False)):
        within(got, value, tol)
    for f, y in ((c.plan.rotate, want), (c.plan.rotate_backward, back)):
        out = (q.clone(), k.clone())
        f(*out, c.positions, out=out)
        assert all(torch.equal(a, b) for a, b in zip(out, y))


@pytest.mark.parametrize("case", [CASES[0], CASES[3]], ids=["halves", "neighbours"])
def test_what_is_not_finite_stays_in_its_pair(case):
    c = Case(*case, positions="near")
    last = c.h - 1
    c.x[0][0, last, 3, 1] = float("nan")                    # in the thread of q's last heads and k's first
    c.x[0][0, 1, 5, 9] = float("inf")
    c.x[1][-1, 0, -1, 2] = float("-inf")
    for got, value in ((c.plan.rotate(*c.on_gpu()[:2], c.positions), c.want(False)), (c.plan.rotate_backward(*c.on_gpu()[:2], c.positions), c.want(True))):
        for y, (want, tol) in zip(got, value):
            within(y, want, tol)
        other = 1 + c.hd // 2 if c.pairs == "half" else 0
        assert torch.isnan(got[0].view(c.b, c.h, c.t, c.hd)[0, last, 3]).nonzero().flatten().tolist() == sorted((1, other))
