"""Attention over prompts beside infinities and NaN: every value that they do not reach keeps the bounds that it has without
them (attention_reference), element by element."""
import numpy as np
import pytest
import torch

import attention_reference as ref
from test_gpu_prompt_attention import Case

pytestmark = pytest.mark.gpu

CASES = [dict(batch=1, tokens=150, heads=2, kvh=1, hd=64), dict(batch=1, tokens=150, heads=2, kvh=1, hd=80, causal=False),
         dict(batch=1, tokens=170, heads=2, kvh=1, hd=128, sequences=4, extents=[3, 40, 90, 90, 160]),
         dict(batch=2, tokens=140, heads=1, kvh=1, hd=64, extents=[100, 37]),
         dict(batch=1, tokens=150, heads=2, kvh=2, hd=256, sequences=2, extents=[0, 77, 150], causal=False),
         dict(batch=1, tokens=290, heads=3, kvh=1, hd=96, sequences=3, extents=[5, 130, 133, 280]),
         dict(batch=1, tokens=150, heads=256, kvh=128, hd=128, extents=[133]),
         dict(batch=1, tokens=150, heads=256, kvh=256, hd=64, sequences=2, extents=[0, 77, 141]),
         # short sequences
         dict(batch=3, tokens=32, heads=2, kvh=1, hd=64), dict(batch=1, tokens=64, heads=512, kvh=256, hd=128, extents=[61])]


@pytest.mark.parametrize("kw", CASES, ids=["_".join(str(x) if not isinstance(x, list) else f"e{sum(x) % 1000}" for x in c.values()) for c in CASES])
@pytest.mark.parametrize("which", ["v", "k", "q", "do"])
def test_what_they_do_not_reach(kw, which):
    print(f"[case] attention {which} {kw}", flush=True)
    c = Case(**kw)
    x = c.do.transpose(1, 2) if which == "do" else getattr(c, which)
    x[0, -1, c.t // 3, 5] = x[0, -1, c.t - 3 * c.t // 10, 2] = x[0, -1, c.t // 2, 7] = float("nan")
    if which == "v":
        x[0, -1, c.t - 3 * c.t // 10, 2], x[0, -1, c.t // 2, 7] = float("inf"), float("-inf")
    outside = np.ones((c.b, c.t), dtype=bool)
    for row, x0, x1 in c.where:
        outside[row, x0:x1] = False
    for y in (c.q, c.k, c.v, c.do.transpose(1, 2)):
        y.transpose(1, 2)[torch.from_numpy(outside)] = float("nan")
    got = c.run()
    reach = ref.not_finite(*(y.double().numpy() for y in (c.q, c.k, c.v)), c.causal, c.scale, c.where, c.do.double().numpy())
    for y in (c.q, c.k, c.v, c.do):
        y[~torch.isfinite(y)] = 0.0
    checked = 0
    for name, (value, bound) in c.want().items():
        fine = np.isfinite(reach[name])
        # the two references agree there
        assert np.abs(reach[name][fine] - value[fine]).max(initial=0.0) <= 1e-9 * max(1.0, np.abs(value[fine]).max(initial=0.0)), name
        err = np.abs(got[name][fine] - value[fine])
        print(f"[attention] {name} {fine.sum()} of {fine.size}, max err/tol {(err / np.maximum(bound[fine], 1e-300)).max(initial=0.0):.3g}", flush=True)
        assert (err <= bound[fine]).all(), name
        checked += int(fine.sum())
    assert checked or which == "k"                          # a NaN in k reaches all that see it: everything, without a mask
