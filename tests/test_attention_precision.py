"""The bar of attention_precision on the CPU: the kernels' roundings pass, the ones that they must not have do not."""
import numpy as np
import pytest

import attention_precision as prec


@pytest.mark.parametrize("n,causal,steep", [(2, True, 1.0), (2, False, 3.0), (8, True, 1.0), (37, True, 1.0), (37, False, 3.0), (300, True, 3.0)])
def test_the_bar_tells_them_apart(n, causal, steep):
    heads, hd = max(8, 2000 // n), 128
    rng = np.random.default_rng(n)
    q, k, v, do = (prec.bf16(rng.standard_normal((heads, n, hd))) for _ in range(4))
    scale = steep * hd ** -0.5
    # 64 bits: ds is not rounded
    x = np.where(np.tril(np.ones((n, n), dtype=bool)) | (not causal), q @ k.transpose(0, 2, 1) * scale, -np.inf)
    p = np.exp(x - x.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    ds = p * (do @ v.transpose(0, 2, 1) - (do * (p @ v)).sum(-1, keepdims=True))
    want = scale * ds @ k, scale * ds.transpose(0, 2, 1) @ q
    for name, mistake in (("none", {}), ("D from the rounded o", dict(d_from_rounded_o=True)), ("ds in one number", dict(ds_in_one=True))):
        shares = [prec.off(prec.bf16(g), w) for g, w in zip(prec.gradients(q, k, v, do, causal, scale, **mistake), want)]
        print(n, causal, steep, name, shares)
        assert all(s <= 1 for s in shares) if not mistake else all(s > 1 for s in shares), name
