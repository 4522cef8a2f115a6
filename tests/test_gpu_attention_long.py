"""Attention over long prompts against its definition in 64 bits: a k/v head and its query heads of each call (the bounds are
derived in attention_reference)."""
import numpy as np
import pytest

import attention_reference as ref
from test_gpu_prompt_attention import Case, check

pytestmark = pytest.mark.gpu

CUTS = sorted(int(x) for x in np.random.default_rng(23).integers(0, 8192, 22))
CASES = [(dict(batch=1, tokens=4096, heads=16, kvh=4, hd=128), 0, 1), (dict(batch=2, tokens=4096, heads=5, kvh=5, hd=64, causal=False, layout="qkv"), 1, 3),
         (dict(batch=1, tokens=8192, heads=32, kvh=8, hd=128, sequences=23, extents=[0, *CUTS, 8192]), 0, 7),
         (dict(batch=1, tokens=8192, heads=8, kvh=8, hd=128), 0, 5), (dict(batch=1, tokens=2999, heads=16, kvh=4, hd=96, causal=False, sequences=2, extents=[0, 2501, 2990]), 0, 2),
         (dict(batch=1, tokens=2100, heads=4, kvh=2, hd=256), 0, 1)]


@pytest.mark.parametrize("kw,row,head", CASES, ids=[f"{c['tokens']}_{c['hd']}_{c['heads']}" for c, _, _ in CASES])
def test_one_head_of_a_long_call(kw, row, head):
    print(f"[case] attention {kw} row {row} k/v head {head}", flush=True)
    c = Case(**kw)
    got = c.run()
    g = c.h // c.kvh
    heads, kv = slice(head * g, head * g + g), slice(head, head + 1)
    one = lambda x, s: x[row:row + 1, s].double().numpy()
    want = ref.attention(one(c.q, heads), one(c.k, kv), one(c.v, kv), c.causal, c.scale, [(0, a, b) for r, a, b in c.where if r == row],
                         c.do[row:row + 1, :, heads].double().numpy())
    part = {"o": got["o"][row:row + 1, :, heads], "lse": got["lse"][row:row + 1, heads], "dq": got["dq"][row:row + 1, heads],
            "dk": got["dk"][row:row + 1, kv], "dv": got["dv"][row:row + 1, kv]}
    check(part, want)
