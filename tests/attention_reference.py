"""Attention over whole prompts by its definition (prompt_attention.h) in 64 bits on the CPU, with the bounds that the
kernels' roundings leave."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
HALF = 2.0 ** -8      # half a step of bf16
LEAST = 2.0 ** -126   # the least number that is not denormal


def spans(batch, tokens, sequences, extents):
    """(batch row, first token, token behind the last) of every sequence."""
    if sequences:
        e = [min(max(x, 0), tokens) for x in extents]
        # offsets that do not ascend cut the tokens between the first and the last one
        cuts = sorted({x for x in e if e[0] <= x <= e[-1]}) if e[0] < e[-1] else []
        return [(0, a, b) for a, b in zip(cuts, cuts[1:])]
    e = [tokens] * batch if extents is None else [min(max(x, 0), tokens) for x in extents]
    return [(i, 0, n) for i, n in enumerate(e)]


def head(q, k, v, causal, scale, do=None):
    """One sequence, one query head: q, k, v, do [n, hd] fp64, everything finite. A dict of (value, bound)."""
    n, hd = q.shape
    see = np.tril(np.ones((n, n), dtype=bool)) if causal else np.ones((n, n), dtype=bool)
    x = np.where(see, q @ k.T * scale, -np.inf)
    top = x.max(1, keepdims=True)
    w = np.exp(x - top)
    total = w.sum(1, keepdims=True)
    w = w / total
    lse = (top + np.log(total))[:, 0]
    o = w @ v
    # a logit: an fp32 sum over hd products, times a rounded factor, beside a maximum that it is at most 2^8 away from
    ax = np.where(see, np.abs(q) @ np.abs(k).T * scale, 0.0)
    dx = (hd + 4) * U * ax.max(1) + 3 * U * np.abs(np.where(see, x, 0.0)).max(1) + 3 * U * np.abs(lse) + 16 * U
    rel = dx + 2.0 ** -21                                     # exp2 in hardware
    # probabilities are rounded to bf16; the sum of those before the rounding carries rel and its own n roundings
    terms = w @ np.abs(v)
    out = {"lse": (lse, rel + (n + 8) * U + 2 * U * np.abs(lse)),
           "o": (o, HALF * np.abs(o) + (HALF + (2 * rel + (2 * n + 16) * U)[:, None]) * terms)}
    if do is None:
        return out
    dp = do @ v.T
    delta = (do * o).sum(1, keepdims=True)
    ds = np.where(see, w * (dp - delta), 0.0)
    # p: the logit's error and that of lse; dp and D: fp32 sums over hd, D of a rounded o
    rp = rel + out["lse"][1]
    ddp = (hd + 2) * U * (np.abs(do) @ np.abs(v).T)
    ddelta = (np.abs(do) * out["o"][1]).sum(1, keepdims=True) + (hd + 2) * U * (np.abs(do) * np.abs(o)).sum(1, keepdims=True)
    dds = np.where(see, w * (rp[:, None] * (np.abs(dp) + np.abs(delta)) + (ddp + ddelta) * (1 + rp[:, None])), 0.0) + (HALF + 3 * U) * np.abs(ds)
    sums = (n + 4) * U
    dwp = w * (rp[:, None] + HALF + 3 * U)
    # numbers below 2^-126 may become 0: a probability (an exponential of fp32), and a ds
    dds = dds + np.where(see, LEAST * (1 + np.abs(dp) + np.abs(delta)), 0.0)
    dwp = dwp + np.where(see, LEAST, 0.0)
    # out of these, sums over tokens; the last rounding is added where heads have been added up
    out["dq"] = (scale * ds @ k, scale * (dds + sums * np.abs(ds)) @ np.abs(k))
    out["dk"] = (scale * ds.T @ q, scale * (dds + sums * np.abs(ds)).T @ np.abs(q))
    out["dv"] = (w.T @ do, (dwp + sums * w).T @ np.abs(do))
    return out


def attention(q, k, v, causal, scale, where, do=None):
    """q [b, H, T, hd], k, v [b, KVH, T, hd], do [b, T, H, hd] fp64; where: spans. {name: (value, bound)}, o [b, T, H, hd],
    lse [b, H, T], gradients shaped like their inputs."""
    b, h, t, hd = q.shape
    kvh = k.shape[1]
    zero = lambda *s: [np.zeros(s), np.zeros(s)]
    out = {"o": zero(b, t, h, hd), "lse": [np.full((b, h, t), -np.inf), np.zeros((b, h, t))]}
    if do is not None:
        out |= {"dq": zero(b, h, t, hd), "dk": zero(b, kvh, t, hd), "dv": zero(b, kvh, t, hd)}
    for row, x0, x1 in where:
        if x0 >= x1:
            continue
        for i in range(h):
            g = i // (h // kvh)
            r = head(q[row, i, x0:x1], k[row, g, x0:x1], v[row, g, x0:x1], causal, scale,
                     None if do is None else do[row, x0:x1, i])
            for e in (0, 1):
                out["o"][e][row, x0:x1, i] = r["o"][e]
                out["lse"][e][row, i, x0:x1] = r["lse"][e]
                if do is not None:
                    out["dq"][e][row, i, x0:x1] = r["dq"][e]
                    out["dk"][e][row, g, x0:x1] += r["dk"][e]
                    out["dv"][e][row, g, x0:x1] += r["dv"][e]
    for name in ("dq", "dk", "dv"):
        if name in out:
            value, bound = out[name]
            bound += (HALF + h // kvh * U) * np.abs(value) + 1e-37
    return {name: tuple(x) for name, x in out.items()}


def not_finite(q, k, v, causal, scale, where, do):
    """Where {name} is NaN, and where infinite: every sum over what is seen alone, one by one (small sizes)."""
    b, h, t, hd = q.shape
    kvh = k.shape[1]
    out = {"o": np.zeros((b, t, h, hd)), "lse": np.full((b, h, t), -np.inf), "dq": np.zeros(q.shape), "dk": np.zeros(k.shape), "dv": np.zeros(v.shape)}
    with np.errstate(all="ignore"):
        for row, x0, x1 in where:
            for i in range(h):
                g = i // (h // kvh)
                for s in range(x0, x1):
                    at = np.arange(x0, s + 1 if causal else x1)
                    qs, ks, vs, ds = q[row, i, s], k[row, g, at], v[row, g, at], do[row, s, i]
                    x = ks @ qs * scale
                    top = x.max()
                    w = np.exp(x - top)
                    lse = top + np.log(w.sum())
                    w = np.exp(x - lse)
                    o = (w[:, None] * vs).sum(0)
                    dsum = w * ((vs * ds).sum(1) - (ds * o).sum())
                    out["o"][row, s, i], out["lse"][row, i, s] = o, lse
                    out["dq"][row, i, s] = (dsum[:, None] * ks).sum(0) * scale
                    out["dk"][row, g, at] += dsum[:, None] * qs * scale
                    out["dv"][row, g, at] += w[:, None] * ds
    return out
