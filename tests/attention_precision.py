"""How far the gradients of attention over whole prompts may be off in the 2-norm (prompt_attention.h): what their own rounding to
bf16 leaves, and next to nothing more.

dq and dk are sums of ds k and ds q with ds = p (dp - D). dp and D are fp32 numbers, D is made from p and dp and not from
an o that was rounded, and ds goes to its products as two bf16 numbers. So what remains is

* each result's rounding: an error of up to half a step h_i of bf16, evenly spread, so that the sum of N of their squares is
  sum h_i^2 / 3, to within 0.9 / sqrt(N) of itself (a standard deviation); 1.1 times its root is ten of these
  from 4000 numbers on;
* ds in two numbers: 2^-16 of it;
* fp32: logits are off by about sqrt(hd) 2^-24 of the sum of their products' sizes, p by as much, and ds by p times that of |dp| + |D|, which
  here are up to some 30 times |ds|: 30 * 12 * 2^-24 * 8 < 2^-12. That covers the line above as well.

D from a rounded o adds 2^-9 / sqrt(3) of |do| |o| to every ds of a row, more than all of it where a row sees few keys."""
from __future__ import annotations

import numpy as np

FEW = 128   # rows that see at most as many keys have their D corrected before dq is made


def half_steps(x):
    """Half of the step of bf16 at x."""
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 8)


def off(got, want):
    """The error's 2-norm as a share of what is allowed."""
    assert want.size >= 4000
    allowed = 1.1 * np.sqrt((half_steps(want) ** 2).sum() / 3) + 2.0 ** -12 * np.sqrt((want ** 2).sum())
    return float(np.sqrt(((got - want) ** 2).sum()) / allowed)


def bf16(x):
    """x rounded to bf16 (ties to even)."""
    bits = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    bits = (bits + 0x7FFF + ((bits >> 16) & 1)) >> 16 << 16
    return bits.astype(np.uint32).view(np.float32).astype(np.float64)


def gradients(q, k, v, do, causal, scale, d_from_rounded_o=False, ds_in_one=False):
    """dq and dk of heads [heads, n, hd] with ds rounded as it is for its products; D exact, or (a mistake) from o as the forward pass
    rounds it."""
    n = q.shape[1]
    x = q @ k.transpose(0, 2, 1) * scale
    if causal:
        x = np.where(np.tril(np.ones((n, n), dtype=bool)), x, -np.inf)
    p = np.exp(x - x.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    o = bf16(bf16(p) @ v) if d_from_rounded_o else p @ v
    ds = p * (do @ v.transpose(0, 2, 1) - (do * o).sum(-1, keepdims=True))
    first = bf16(ds)
    ds = first if ds_in_one else first + bf16(ds - first)
    return scale * ds @ k, scale * ds.transpose(0, 2, 1) @ q
