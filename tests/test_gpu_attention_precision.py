"""dq and dk of attention over prompts are off by no more than their own rounding (attention_precision has the bar)."""
import numpy as np
import pytest
import torch

import attention_precision as prec
from test_gpu_prompt_attention import Case

pytestmark = pytest.mark.gpu

# every shape of workgroup, rows that see one key to hundreds, sequences side by side in a workgroup; steep: the logits' spread
CASES = [dict(batch=64, tokens=2, heads=4, kvh=2, hd=128), dict(batch=64, tokens=2, heads=4, kvh=4, hd=64, causal=False, steep=3.0),
         dict(batch=16, tokens=8, heads=4, kvh=4, hd=128), dict(batch=8, tokens=30, heads=8, kvh=2, hd=256), dict(batch=16, tokens=30, heads=8, kvh=8, hd=40, steep=3.0),
         dict(batch=1, tokens=37, heads=8, kvh=8, hd=128), dict(batch=1, tokens=37, heads=8, kvh=2, hd=96, causal=False, steep=3.0),
         dict(batch=8, tokens=50, heads=64, kvh=64, hd=64), dict(batch=8, tokens=60, heads=64, kvh=16, hd=128, causal=False, steep=3.0),
         dict(batch=2, tokens=130, heads=8, kvh=2, hd=192), dict(batch=1, tokens=200, heads=4, kvh=4, hd=256, causal=False, steep=3.0),
         dict(batch=2, tokens=200, heads=4, kvh=2, hd=64, steep=3.0), dict(batch=2, tokens=250, heads=128, kvh=64, hd=128, steep=3.0),
         dict(batch=2, tokens=250, heads=128, kvh=128, hd=72, causal=False, extents=[250, 101]), dict(batch=1, tokens=520, heads=4, kvh=1, hd=128),
         dict(batch=1, tokens=512, heads=2, kvh=2, hd=64, steep=3.0), dict(batch=1, tokens=300, heads=4, kvh=4, hd=128, causal=False, steep=3.0),
         # short sequences behind long ones: their first rows share a workgroup with rows that see many keys
         dict(batch=1, tokens=700, heads=4, kvh=2, hd=128, sequences=5, extents=[3, 460, 470, 471, 600, 690], steep=3.0),
         dict(batch=1, tokens=700, heads=4, kvh=2, hd=64, sequences=5, extents=[3, 460, 470, 471, 600, 690], causal=False, steep=3.0),
         dict(batch=1, tokens=700, heads=4, kvh=4, hd=136, sequences=4, extents=[0, 420, 430, 500, 700], steep=3.0),
         dict(batch=1, tokens=1030, heads=128, kvh=64, hd=64, sequences=9, extents=[0, 2, 5, 300, 310, 640, 650, 655, 1000, 1030], steep=3.0)]


@pytest.mark.parametrize("kw", CASES, ids=["_".join(str(x) if not isinstance(x, list) else f"e{sum(x) % 1000}" for x in c.values()) for c in CASES])
def test_gradients_to_their_rounding(kw):
    print(f"[case] attention {kw}", flush=True)
    kw = dict(kw)
    steep = kw.pop("steep", 1.0)
    c = Case(**kw, scale=steep * kw["hd"] ** -0.5)
    got, want = c.run(), c.want()
    # where logits are steep D's error reaches dq in rows that see many keys
    rows = np.zeros((c.b, c.t), dtype=bool)
    for b, x0, x1 in c.where:
        seen = np.arange(1, x1 - x0 + 1) if c.causal else np.full(x1 - x0, x1 - x0)
        rows[b, x0:x1] = (seen <= prec.FEW) | (steep == 1.0)
    at = np.broadcast_to(rows[:, None, :], want["dq"][0].shape[:3])
    shares = {"dk": prec.off(got["dk"], want["dk"][0])}
    if at.any():
        shares["dq"] = prec.off(got["dq"][at], want["dq"][0][at])
    print(f"[attention] norm err/tol {shares}", flush=True)
    assert max(shares.values()) <= 1
