"""The key/value cache's definition (kv_cache.h) in NumPy and torch on the CPU: the stored bytes bit for bit, and the
attention in 64 bits with the bound that the kernels' roundings leave."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24


def bf16_bits(f32: np.ndarray) -> np.ndarray:
    """The upper halves of fp32 numbers whose lower halves are 0."""
    return (np.ascontiguousarray(f32, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def quantise(x: torch.Tensor, bits: int):
    """(codes, scale, zero) of bf16 rows: uint8 [..., hd], fp32 [...], fp32 [...]."""
    f = x.float().numpy()
    most = np.float32(2 ** bits - 1)
    with np.errstate(all="ignore"):
        zero = f.min(-1)
        step = (f.max(-1) - zero) / most                                 # fp32, as the definition says
        # the least bfloat16 number not below it
        scale = ((step.view(np.uint32).astype(np.uint64) + 0xFFFF) & 0xFFFF0000).astype(np.uint32).view(np.float32)
        kept = scale <= np.float32(2.0 ** 24)
        code = np.rint((f - zero[..., None]) / scale[..., None])
        code = np.where((kept & (scale > 0))[..., None], np.minimum(code, most), 0).astype(np.uint8)
    return code, np.where(kept, scale, np.float32(np.nan)), np.where(kept, zero, np.float32(np.nan))


def pack(code: np.ndarray, bits: int) -> np.ndarray:
    return code if bits == 8 else (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def positions(length: int, count: int | None, tokens: int, capacity: int):
    """{token of the step: position} of a sequence's real tokens with a place in the cache."""
    count = tokens if count is None else min(max(count, 0), tokens)
    first = max(length, 0) - count
    return {s: first + s for s in range(count) if 0 <= first + s < capacity}


def attend(q, k_rows, v_rows, own, length, group, scale, bits):
    """One sequence. q [H, T, hd] fp64; k_rows, v_rows: (code, scale, zero) [KVH, positions, ...] fp64 with a scale of -1
    where there is no page; own {token: position}; returns (o, tolerance) [T, H, hd]."""
    H, T, hd = q.shape
    o, tol = np.zeros((T, H, hd)), np.zeros((T, H, hd))
    for s, p in own.items():
        for h in range(H):
            kc, ks, kz = (a[h // group][:min(p + 1, length)] for a in k_rows)
            vc, vs, vz = (a[h // group][:min(p + 1, length)] for a in v_rows)
            at = ks != -1
            if not at.any():
                continue
            kc, ks, kz, vc, vs, vz = (a[at] for a in (kc, ks, kz, vc, vs, vz))
            with np.errstate(all="ignore"):
                x = (ks * (kc @ q[h, s]) + kz * q[h, s].sum()) * scale
                w = np.exp(x - x.max()) if np.isfinite(x).all() else np.full(x.shape, np.nan)
                w = w / w.sum()
                o[s, h] = (w * vs) @ vc + (w * vz).sum()
                # a logit: its fp32 sums over hd terms and a few products, held beside a maximum and 80
                aq = np.abs(q[h, s])
                dx = (hd + 8) * U * scale * (ks * (kc @ aq) + np.abs(kz) * aq.sum()) * 2 + U * (3 * np.abs(x).max() + 200)
                # exp2 in hardware: 2^-22; numerator and denominator each carry the relative error of p
                rel = 2 * (dx.max() + 2.0 ** -21)
                terms = (w * vs) @ vc + (w * np.abs(vz)).sum()
                # The kernel sums b (c - C) + p (z + C s) with b = p s rounded to bf16 and C the middle code: b = p s (1 + d),
                # |d| <= 2^-8 (half a step), so the sum is off by d p s (c - C) a position. Both sums, and C sum b apart, are
                # fp32 sums of terms of up to p s (c + C) + p |z|. One last rounding.
                mid = (2 ** bits - 1) / 2
                off = (w * vs) @ np.abs(vc - mid)
                terms = terms + 2 * mid * (w * vs).sum()
                tol[s, h] = 2.0 ** -8 * np.abs(o[s, h]) + 2.0 ** -8 * off + (rel + (len(x) + 40) * U) * terms
    return o, tol
