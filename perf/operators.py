"""The operators on either side of the fused input projection, as a program calls them, with their plain forms.

A transformer block normalises its input, projects it (FusedProjection), keeps k and v in a cache and attends over
that cache. Here are the steps around the projection:

  norm       layer norm over the channels of a channels-first or token-major activation
  norm_grad  its backward pass: dx, dgamma and dbeta
  store      quantises k and v into a paged cache of 4 or 8 bits and reads the stored values back
  attend     attention of the step's queries over such a cache, from one token to a prompt's chunk

`run` takes the plain form (elementary torch operations in 32 bits, rounded once) unless `own` is set; then it makes
the calls of the framework. `exact` has the same results in 64 bits.

The cache's format: a row is the head_dim values of one token of one k/v head. zero is the row's least value, scale the
least bfloat16 number not below (greatest - least) / (2^bits - 1), both kept in bfloat16; a value's code is
(value - zero) / scale rounded to the nearest whole number (ties to even; 0 where scale is 0) and at most 2^bits - 1.
It stands for zero + scale * code. Codes lie in [pages, kv_heads, page_size, head_dim * bits / 8] bytes (at 4 bits the
even element in the low half), scale and zero in [pages, kv_heads, page_size, 2]. Position p of sequence i is slot
p % page_size of page table[i, p // page_size]. A step has up to `tokens` tokens in each sequence, counts[i] of them
real; they are the last of the lengths[i] that the cache holds after it.
"""
import math

import torch

own = False
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases
def _norm(name, op, layout, dtype, batch, channels, tokens, pad=0):
    return {"name": name, "op": op, "layout": layout, "dtype": dtype, "batch": batch, "channels": channels,
            "tokens": tokens, "pad": pad}


def _cache(name, op, bits, batch, tokens, heads, kv_heads, head_dim, page, longest, ragged=True, empty=False):
    return {"name": name, "op": op, "bits": bits, "batch": batch, "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "longest": longest, "ragged": ragged,
            "empty": empty}


def listed():
    return [
        # one decoding step of the decoder's width: 16 sequences, one token each
        _norm("norm_step", "norm", "tokens_last", "bf16", 16, 4096, 1),
        # the Walrus activation, normalised over its channels where it lies
        _norm("norm_walrus", "norm", "channels_first", "bf16", 24, 768, 1024),
        # a prompt in 32 bits, its rows cut out of wider ones, the width no multiple of anything
        _norm("norm_f32_odd", "norm", "tokens_last", "f32", 3, 1387, 1021, pad=5),
        # a BERT batch in training
        _norm("norm_grad_bert", "norm_grad", "tokens_last", "bf16", 32, 768, 512),
        # the wider Walrus activation in training
        _norm("norm_grad_walrus", "norm_grad", "channels_first", "bf16", 24, 1408, 1024),
        # a training batch in 32 bits with an odd number of grid points
        _norm("norm_grad_f32_odd", "norm_grad", "channels_first", "f32", 6, 320, 1847),
        # one decoding step's k and v: 16 sequences, one token each
        _cache("store_step", "store", 4, 16, 1, 32, 8, 128, 64, 4096),
        # the prompts of four sequences, padded to the longest, in 8 bits
        _cache("store_prompt", "store", 8, 4, 2048, 12, 12, 64, 16, 2048),
        # a single conversation's decoding step
        _cache("attend_step_one", "attend", 4, 1, 1, 32, 8, 128, 64, 1023),
        # a loaded server's decoding step: sequences of all lengths, one slot of the batch unused
        _cache("attend_step_many", "attend", 4, 64, 1, 32, 8, 128, 64, 8191, empty=True),
        # plain multi-head attention over 8 bits, a few drafted tokens at a time
        _cache("attend_draft_8bit", "attend", 8, 24, 5, 12, 12, 64, 16, 3333),
        # a chunk of a long prompt
        _cache("attend_chunk", "attend", 4, 2, 1024, 32, 8, 128, 64, 4096),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "store", "attend", "attend"])
    if op in ("norm", "norm_grad"):
        layout = rng.choice(["channels_first", "tokens_last"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        channels = _spread(rng, 16, 2048 if layout == "channels_first" else 12288)
        if rng.random() < 0.7:
            channels = -(-channels // 8) * 8
        most = (24 * 1408 * 1024 if dtype == "bf16" else 6 * 1408 * 1024) // channels
        rows = _spread(rng, 1, most)
        batch = _spread(rng, 1, min(rows, 64))
        tokens = max(1, rows // batch)
        if tokens >= 8 and rng.random() < 0.7:
            tokens -= tokens % 8
        return _norm_free(op, layout, dtype, batch, channels, tokens, rng.choice([0, 0, 8, 3]))
    bits = rng.choice([4, 4, 8])
    head_dim = rng.choice([32, 64, 64, 96, 128, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 12])
    group = rng.choice([1, 1, 2, 4, 6, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "store":
        tokens = rng.choice([1, 1, _spread(rng, 2, 2048)])
        batch = _spread(rng, 1, max(1, min(64, 8192 // tokens)))
        longest = tokens + rng.choice([0, _spread(rng, 1, 4096)])
    else:
        tokens = rng.choice([1, 1, _spread(rng, 2, 16), _spread(rng, 17, 1024)])
        longest = max(tokens, _spread(rng, 16, 32768 if tokens <= 16 else 4096))
        cells = 64 * 8 * 8191 * 128 // 2                     # cached values of a side
        work = 2 * 32 * 1024 * 4096 * 128                    # products of queries and keys
        most = min(cells // (kv_heads * longest * head_dim), work // (kv_heads * group * tokens * longest * head_dim))
        batch = _spread(rng, 1, max(1, min(64, most)))
        while tokens > 1 and kv_heads * group * tokens * longest * head_dim * batch > work:
            tokens = max(1, tokens // 2)
    case = _cache("", op, bits, batch, tokens, kv_heads * group, kv_heads, head_dim, page, longest,
                  rng.random() < 0.7, batch > 1 and rng.random() < 0.3)
    del case["name"]
    return case


def _norm_free(*a):
    case = _norm("", *a)
    del case["name"]
    return case


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (_prepare_norm if case["op"] in ("norm", "norm_grad") else _prepare_cache)(case, g)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _prepare_norm(case, g):
    b, c, t, pad, dtype = case["batch"], case["channels"], case["tokens"], case["pad"], TYPES[case["dtype"]]
    first = case["layout"] == "channels_first"
    # activations have a few channels far wider and further off than the rest
    wide = 1.0 + 9.0 * (torch.rand(c, generator=g, device=DEV) < 0.02).float()
    off = 0.5 * _randn(g, c) * wide
    if first:
        x = (_randn(g, b, c + pad, t)[:, :c] * wide[:, None] + off[:, None]).to(dtype)
        if pad:
            x = torch.cat([x, x[:, :1].expand(b, pad, t)], 1)[:, :c]
    else:
        x = (_randn(g, b, t, c) * wide + off).to(dtype)
        if pad:
            x = torch.cat([x, x[..., :1].expand(b, t, pad)], 2)[..., :c]
    s = {"op": case["op"], "first": first, "eps": 1e-5, "x": x, "gamma": (1.0 + 0.2 * _randn(g, c)).to(dtype),
         "beta": (0.1 * _randn(g, c)).to(dtype)}
    if case["op"] == "norm_grad":
        rows = _rows(x, first).float()
        mean = rows.mean(-1)
        s["stats"] = torch.stack([mean, (rows.var(-1, unbiased=False) + s["eps"]).rsqrt()])
        s["dy"] = _randn(g, *x.shape).to(dtype)
    if own:
        from ff_input_projection_amd import LayerNorm
        s["plan"] = LayerNorm.for_tensor(x, case["layout"], eps=s["eps"], has_bias=True)
    return s


def _prepare_cache(case, g):
    b, t, kvh, hd, page, longest = (case[k] for k in ("batch", "tokens", "kv_heads", "head_dim", "page", "longest"))
    max_pages = -(-longest // page)
    n_pages = b * max_pages + 3
    table = torch.randperm(n_pages, generator=g, device=DEV)[:b * max_pages].view(b, max_pages).to(torch.int32)
    lengths = torch.full((b,), longest, device=DEV, dtype=torch.int64)
    counts = torch.full((b,), t, device=DEV, dtype=torch.int64)
    if case["ragged"]:
        share = torch.rand((b,), generator=g, device=DEV)
        share[0] = 1.0
        lengths = (longest * (0.3 + 0.7 * share)).round().long().clamp(1, longest)
        counts = torch.minimum((t * (0.5 + 0.5 * share)).round().long().clamp(min=1), lengths)
    if case["empty"]:
        lengths[-1] = 0
        counts[-1] = 0
    table = table.masked_fill(torch.arange(max_pages, device=DEV) >= (lengths[:, None] + page - 1) // page, -1)
    s = {"op": case["op"], "bits": case["bits"], "tokens": t, "heads": case["heads"], "kv_heads": kvh, "head_dim": hd,
         "page": page, "table": table.contiguous(), "lengths": lengths.to(torch.int32), "counts": counts.to(torch.int32)}
    # a few channels of the keys are far off, as rotated keys' slow channels are
    k_off = 2.0 * _randn(g, kvh, 1, hd) * (torch.rand((hd,), generator=g, device=DEV) < 0.06)
    if case["op"] == "store":
        s["storage"] = (torch.zeros((n_pages, kvh, page, hd * case["bits"] // 8), device=DEV, dtype=torch.uint8),
                        torch.zeros((n_pages, kvh, page, 2), device=DEV, dtype=torch.bfloat16),
                        torch.zeros((n_pages, kvh, page, hd * case["bits"] // 8), device=DEV, dtype=torch.uint8),
                        torch.zeros((n_pages, kvh, page, 2), device=DEV, dtype=torch.bfloat16))
        s["k"] = (_randn(g, b, kvh, t, hd) + k_off).to(torch.bfloat16).view(b * kvh, t, hd)
        s["v"] = _randn(g, b * kvh, t, hd).to(torch.bfloat16)
    else:
        k = _quantise((_randn(g, n_pages, kvh, page, hd) + k_off).to(torch.bfloat16), case["bits"])
        v = _quantise(_randn(g, n_pages, kvh, page, hd).to(torch.bfloat16), case["bits"])
        s["storage"] = k + v
        s["q"] = _randn(g, b * case["heads"], t, hd).to(torch.bfloat16)
    if own:
        from ff_input_projection_amd import KVCache
        s["plan"] = KVCache(b, t, case["heads"], hd, n_kv_heads=kvh, bits=case["bits"], page_size=page,
                            n_pages=n_pages, max_pages=max_pages)
        if case["op"] == "attend":
            s["workspace"] = s["plan"].alloc_workspace(DEV)
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    return {"norm": _run_norm, "norm_grad": _run_norm_grad, "store": _run_store, "attend": _run_attend}[state["op"]](state)


def _rows(x, first):
    """[tokens, channels] of an activation."""
    return x.transpose(1, 2).reshape(-1, x.shape[1]) if first else x.reshape(-1, x.shape[2])


def _back(rows, x, first):
    """The activation, laid out like x, of its rows."""
    if first:
        return rows.view(x.shape[0], x.shape[2], x.shape[1]).transpose(1, 2).contiguous()
    return rows.view(x.shape)


def _run_norm(s):
    if own:
        return s["plan"](s["x"], s["gamma"], s["beta"])
    x = _rows(s["x"], s["first"]).float()
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    rstd = 1.0 / ((d * d).mean(-1, keepdim=True) + s["eps"]).sqrt()
    y = d * rstd * s["gamma"].float() + s["beta"].float()
    return _back(y.to(s["x"].dtype), s["x"], s["first"]), torch.stack([mean[:, 0], rstd[:, 0]])


def _run_norm_grad(s):
    if own:
        return s["plan"].backward(s["x"], s["gamma"], s["stats"], s["dy"])
    dtype, first = s["x"].dtype, s["first"]
    dy = _rows(s["dy"], first).float()
    xhat = (_rows(s["x"], first).float() - s["stats"][0][:, None]) * s["stats"][1][:, None]
    dg = dy * s["gamma"].float()
    dx = s["stats"][1][:, None] * (dg - dg.mean(-1, keepdim=True) - xhat * (dg * xhat).mean(-1, keepdim=True))
    # sums over many tokens: in 64 bits
    dgamma = (dy * xhat).sum(0, dtype=torch.float64)
    dbeta = dy.sum(0, dtype=torch.float64)
    return _back(dx.to(dtype), s["x"], first), dgamma.to(dtype), dbeta.to(dtype)


def _quantise(x, bits):
    """(codes in bytes, scale and zero) of rows along the last dimension."""
    x = x.float()
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    most = torch.full_like(low, 2 ** bits - 1)
    # up to the next bfloat16 number: the bits of a number >= 0 are ordered as it is
    scale = ((((high - low) / most).view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)
    codes = torch.where(scale > 0, (x - low) / scale, 0.0).round().clamp(max=2 ** bits - 1).to(torch.uint8)
    if bits == 4:
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return codes.contiguous(), torch.cat([scale, low], -1).to(torch.bfloat16)


def _values(codes, params, bits, dtype=torch.float32):
    """What stored rows stand for."""
    if bits == 4:
        codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    params = params.to(dtype)
    return params[..., 1:] + params[..., :1] * codes.to(dtype)


def _where(s):
    """(page, slot, sequence, token) of each real token of the step."""
    at = torch.arange(s["tokens"], device=DEV)
    position = (s["lengths"] - s["counts"])[:, None] + at
    seq, tok = ((at < s["counts"][:, None]) & (position >= 0)).nonzero(as_tuple=True)
    position = position[seq, tok]
    return s["table"][seq, position // s["page"]].long(), position % s["page"], seq, tok


def _run_store(s):
    if own:
        s["plan"].write(s["storage"], s["k"], s["v"], s["table"], s["lengths"], s["counts"])
        return s["plan"].read(s["storage"], s["table"], s["lengths"], s["counts"])
    page, slot, seq, tok = _where(s)
    b, kvh, t, hd = s["table"].shape[0], s["kv_heads"], s["tokens"], s["head_dim"]
    out = []
    for x, codes, params in ((s["k"], *s["storage"][:2]), (s["v"], *s["storage"][2:])):
        codes[page, :, slot], params[page, :, slot] = _quantise(x.view(b, kvh, t, hd)[seq, :, tok], s["bits"])
        back = torch.zeros((b, kvh, t, hd), device=DEV, dtype=torch.bfloat16)
        back[seq, :, tok] = _values(codes[page, :, slot], params[page, :, slot], s["bits"]).to(torch.bfloat16)
        out.append(back.view(b * kvh, t, hd))
    return tuple(out)


def _pages(s, codes, params, dtype):
    """[sequences, kv_heads, positions, head_dim]: the cached values in order (0 where there are none)."""
    b, n = s["table"].shape
    at = s["table"].clamp(min=0).long()
    x = _values(codes[at], params[at], s["bits"], dtype)
    return x.transpose(1, 2).reshape(b, s["kv_heads"], n * s["page"], s["head_dim"])


def _run_attend(s):
    if own:
        return s["plan"].attend(s["storage"], s["q"], s["table"], s["lengths"], s["counts"], workspace=s["workspace"])
    b, h, kvh, t, hd = s["table"].shape[0], s["heads"], s["kv_heads"], s["tokens"], s["head_dim"]
    k, v = (_pages(s, *s["storage"][i:i + 2], torch.float32) for i in (0, 2))
    q = s["q"].float().view(b, kvh, h // kvh * t, hd)
    logits = (k @ q.transpose(-1, -2).contiguous()).view(b, kvh, -1, h // kvh, t) * hd ** -0.5
    at = torch.arange(t, device=DEV)
    last = (s["lengths"] - s["counts"])[:, None] + at                                  # a query's own position
    seen = torch.arange(k.shape[2], device=DEV)[:, None] <= last[:, None, :]           # [b, positions, t]
    seen = seen & (at < s["counts"][:, None])[:, None, :]
    logits = logits.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = logits.amax(2, keepdim=True).clamp(min=-3e38)
    p = (logits - top).exp()
    total = p.sum(2)                                                                   # [b, kvh, group, t]
    o = (p.flatten(3).transpose(-1, -2) @ v).view(b, kvh, h // kvh, t, hd)
    o = o / torch.where(total > 0, total, 1.0)[..., None]
    return o.view(b, h, t, hd).transpose(1, 2).reshape(b, t, h * hd).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    if case["op"] in ("norm", "norm_grad"):
        n, size = case["batch"] * case["tokens"] * case["channels"], 2 if case["dtype"] == "bf16" else 4
        sides = 2 if case["op"] == "norm" else 3
        return {"bytes": sides * n * size + 8 * case["batch"] * case["tokens"] + sides * case["channels"] * size,
                "flops": (8 if case["op"] == "norm" else 14) * n}
    b, t, kvh, hd, bits = (case[k] for k in ("batch", "tokens", "kv_heads", "head_dim", "bits"))
    row = hd * bits / 8 + 4
    shares = ([1.0] + [0.65] * (b - 1) if case["ragged"] else [1.0] * b)[:b - 1 if case["empty"] else b]
    if case["op"] == "store":
        n = sum(0.5 + 0.5 * (x - 0.3) / 0.7 for x in shares) * t * kvh * 2 if case["ragged"] else len(shares) * t * kvh * 2
        # the real rows in, their codes written and read, the whole padded block of values out
        return {"bytes": n * (2 * hd + 2 * row) + 2 * b * kvh * t * 2 * hd, "flops": 8 * n * hd}
    cached = sum(shares) * case["longest"]
    seen = sum(max(x * case["longest"] - t / 2, t / 2) for x in shares)
    return {"bytes": cached * kvh * 2 * row + 2 * b * t * case["heads"] * hd * 2,
            "flops": 4 * seen * t * case["heads"] * hd}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "store": _exact_store, "attend": _exact_attend}[case["op"]](s)


def _exact_norm(s):
    axis = 1 if s["first"] else 2
    wide = [1, -1, 1] if s["first"] else [1, 1, -1]
    x = s["x"].double()
    mean = x.mean(axis, keepdim=True)
    var = (x - mean).square().mean(axis, keepdim=True)
    rstd = (var + s["eps"]) ** -0.5
    y = (x - mean) * rstd * s["gamma"].double().view(wide) + s["beta"].double().view(wide)
    return y, torch.stack([mean.reshape(-1), rstd.reshape(-1)])


def _exact_norm_grad(s):
    """By the chain rule through y = gamma (x - mean) rstd + beta, mean and rstd functions of x."""
    axis, other = (1, (0, 2)) if s["first"] else (2, (0, 1))
    wide = [1, -1, 1] if s["first"] else [1, 1, -1]
    x, dy = s["x"].double(), s["dy"].double()
    keep = [x.shape[0], 1, x.shape[2]] if s["first"] else [x.shape[0], x.shape[1], 1]
    mean, rstd = s["stats"][0].double().view(keep), s["stats"][1].double().view(keep)
    centred = x - mean
    dn = dy * s["gamma"].double().view(wide)
    d_rstd = (dn * centred).sum(axis, keepdim=True)
    d_var = -0.5 * d_rstd * rstd ** 3
    d_centred = dn * rstd + 2.0 * d_var * centred / x.shape[axis]
    dx = d_centred - d_centred.mean(axis, keepdim=True)
    # the centred values sum to the rounding of the given mean alone: that term is no part of the definition
    dx = dx + (2.0 * d_var * centred / x.shape[axis]).mean(axis, keepdim=True)
    return dx, (dy * centred * rstd).sum(other), dy.sum(other)


def _exact_store(s):
    b, kvh, t, hd = s["table"].shape[0], s["kv_heads"], s["tokens"], s["head_dim"]
    most = 2 ** s["bits"] - 1
    real = (torch.arange(t, device=DEV) < s["counts"][:, None])[:, None, :, None]
    out = []
    for x in (s["k"], s["v"]):
        x = x.double().view(b, kvh, t, hd)
        low = x.min(-1, keepdim=True).values
        step = (x.max(-1, keepdim=True).values - low) / most
        near = step.to(torch.bfloat16)
        above = (near.view(torch.int16) + 1).view(torch.bfloat16)
        step = torch.where(near.double() < step, above, near).double()
        code = torch.where(step > 0, ((x - low) / step).round().clamp(max=most), 0.0)
        out.append(torch.where(real, low + step * code, 0.0).view(b * kvh, t, hd))
    return tuple(out)


def _exact_attend(s):
    b, h, kvh, t, hd = s["table"].shape[0], s["heads"], s["kv_heads"], s["tokens"], s["head_dim"]
    group = h // kvh
    out = torch.zeros((b, t, h, hd), device=DEV, dtype=torch.float64)
    q = s["q"].double().view(b, h, t, hd)
    for i, (length, count) in enumerate(zip(s["lengths"].tolist(), s["counts"].tolist())):
        if count == 0:
            continue
        at = torch.arange(length, device=DEV)
        page, slot = s["table"][i, at // s["page"]].long(), at % s["page"]
        own_at = torch.arange(length - count, length, device=DEV)
        late = at[None, :] > own_at[:, None]
        for j in range(kvh):
            k, v = (_values(s["storage"][n][page, j, slot], s["storage"][n + 1][page, j, slot], s["bits"],
                            torch.float64) for n in (0, 2))
            x = torch.matmul(q[i, j * group:(j + 1) * group, :count], k.t().contiguous()) / math.sqrt(hd)
            x = x.masked_fill(late, -math.inf).softmax(-1)
            out[i, :count, j * group:(j + 1) * group] = torch.matmul(x, v).transpose(0, 1)
    return out.view(b, t, h * hd)
