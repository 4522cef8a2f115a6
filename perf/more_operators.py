"""Rotary positions and attention over whole prompts, as a program calls them, with their plain forms.

Between the fused projection and the projection of the attention's output, in training and for prompts:

  rope         splits a projected qkv into heads and rotates q and k by each token's position, or rotates
               head-major q and k
  rope_grad    its backward pass
  prompt       attention of whole sequences over themselves: a padded batch or packed sequences, causal or not,
               grouped heads; o and the logarithm of each row's sum of exponentials
  train        the same, then its gradients dq, dk and dv

`run` takes the plain form (elementary torch operations in 32 bits, angles in 64, rounded once) unless `own` is set;
then it makes the calls of the framework. `exact` has the same results in 64 bits.

Angles: pair i of a rotated width of `dims` turns by theta_i = base^(-2i/dims) a position. Scaled "linear" it is
theta_i / factor. Scaled "by_parts", with r_i = ORIGINAL theta_i / (2 pi) turns over the original length and
g = min(max((r_i - 1) / (32 - 1), 0), 1), it is theta_i (g + (1 - g) / factor), and the rotated elements are multiplied
by 0.1 ln(factor) + 1. Pair i is elements i and i + dims / 2 ("half") or 2i and 2i + 1 ("interleaved") of a head.
"""
import math
import random

import torch

own = False
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BASE, ORIGINAL, LOW, HIGH = 10000.0, 4096, 1.0, 32.0


# ------------------------------------------------------------------------------------------------ cases
def _rope(name, op, form, dtype, batch, tokens, heads, kv_heads, head_dim, dims, pairs, order="contiguous",
          scaling="none", factor=1.0, furthest=4095):
    return {"name": name, "op": op, "form": form, "dtype": dtype, "batch": batch, "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "dims": dims, "pairs": pairs, "order": order,
            "scaling": scaling, "factor": factor, "furthest": furthest}


def _attention(name, op, form, batch, tokens, heads, kv_heads, head_dim, causal, sequences=0, ragged=False):
    return {"name": name, "op": op, "form": form, "batch": batch, "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "causal": causal, "sequences": sequences, "ragged": ragged}


def listed():
    return [
        # a server's decoding step: 16 sequences, each one token at a position of its own
        _rope("rope_step", "rope", "qkv", "bf16", 16, 1, 32, 8, 128, 128, "half", furthest=8191),
        # the decoder's prompts, stretched to eight times the length that it was made for
        _rope("rope_prompt", "rope", "qkv", "bf16", 2, 4096, 32, 32, 128, 128, "half", scaling="by_parts", factor=8.0,
              furthest=32767),
        # the backward pass of the grouped block of 16 heads in 4 groups, 8 of 32 elements rotated
        _rope("rope_grad_gqa", "rope_grad", "qkv", "bf16", 2, 1024, 16, 4, 32, 8, "half", "grouped"),
        # q and k in 32 bits as the projection splits them, neighbouring elements paired, an odd number of tokens
        _rope("rope_grad_f32_odd", "rope_grad", "heads", "f32", 3, 1021, 12, 12, 80, 64, "interleaved",
              scaling="linear", factor=4.0, furthest=16383),
        # one short question
        _attention("prompt_short", "prompt", "heads", 1, 37, 32, 8, 128, True),
        # a server's queue of prompts, packed one behind the other
        _attention("prompt_packed", "prompt", "heads", 1, 8192, 32, 8, 128, True, sequences=23),
        # one long document
        _attention("prompt_long", "prompt", "heads", 1, 8192, 32, 8, 128, True),
        # image tokens attending to each other: 4096 of them, 5 heads, q, k and v side by side in one tensor
        _attention("prompt_image", "prompt", "qkv", 2, 4096, 5, 5, 64, False),
        # the decoder in training
        _attention("train_decoder", "train", "heads", 2, 4096, 32, 8, 128, True),
        # a BERT batch in training, padded to its longest sentence
        _attention("train_bert", "train", "heads", 32, 512, 12, 12, 64, False, ragged=True),
        # the grouped block, its batch packed, an odd number of tokens
        _attention("train_packed_odd", "train", "heads", 1, 2999, 16, 4, 96, True, sequences=7),
        # a small batch in training: the Walrus grid's 1024 points, one step
        _attention("train_small", "train", "qkv", 1, 1024, 12, 12, 64, False),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_grad", "prompt", "prompt", "train", "train"])
    head_dim = rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 12])
    heads = kv_heads * rng.choice([1, 1, 2, 4, 6])
    if op in ("rope", "rope_grad"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 2 * 4096 * 96 * 128 // (1 if dtype == "bf16" else 2) // ((heads + 2 * kv_heads) * head_dim)
        rows = _spread(rng, 1, most)
        batch = _spread(rng, 1, min(rows, 64))
        scaling = rng.choice(["none", "linear", "by_parts"])
        factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0])
        case = _rope("", op, rng.choice(["qkv", "qkv", "heads"]), dtype, batch, max(1, rows // batch), heads, kv_heads,
                     head_dim, rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4]),
                     rng.choice(["half", "interleaved"]), rng.choice(["contiguous", "grouped"]), scaling, factor,
                     int(_spread(rng, 256, 4096) * factor))
        if case["form"] == "heads":
            case["order"] = "contiguous"
    else:
        work = (32 * 8192 ** 2 if op == "prompt" else 2 * 32 * 4096 ** 2) * 128
        # in training two tokens at least: one alone has gradients of 0, for q and k, of which only roundings are left
        tokens = _spread(rng, 1 if op == "prompt" else 2, 8192)
        while heads * tokens ** 2 * head_dim > work:
            tokens = tokens * 2 // 3
        batch = _spread(rng, 1, max(1, min(64, work // (heads * tokens ** 2 * head_dim))))
        while batch > 1 and batch * tokens * heads * head_dim > 8192 * 32 * 128:
            batch //= 2
        sequences = 0
        if rng.random() < 0.5:
            tokens, batch = min(8192, batch * tokens), 1
            while heads * tokens ** 2 * head_dim > work:
                tokens = tokens * 2 // 3
            sequences = _spread(rng, 1, max(1, min(64, tokens // 4)))
        case = _attention("", op, rng.choice(["heads", "heads", "qkv"]), batch, tokens, heads, kv_heads, head_dim,
                          rng.random() < 0.7, sequences, rng.random() < 0.5)
    del case["name"]
    return case


def _extents(case):
    """A padded batch's lengths, or the packed sequences' offsets; None where all are as long as the padding."""
    rng = random.Random(case["tokens"] * 1000 + case["sequences"] * 64 + case["batch"])
    t, n = case["tokens"], case["sequences"]
    if n:
        end = t - (t // 50 if case["ragged"] else 0)          # a few tokens behind the last sequence are no one's
        return [0] + sorted(int(end * rng.random()) for _ in range(n - 1)) + [end]
    if case["ragged"]:
        return [max(1, round(t * (0.2 + 0.8 * rng.random()))) for _ in range(case["batch"] - 1)] + [t]
    return None


def _spans(case):
    """(batch row, first token, token behind the last) of every sequence."""
    e = _extents(case)
    if case["sequences"]:
        return [(0, a, b) for a, b in zip(e, e[1:])]
    return [(i, 0, case["tokens"] if e is None else e[i]) for i in range(case["batch"])]


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (_prepare_rope if case["op"] in ("rope", "rope_grad") else _prepare_attention)(case, g)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _frequencies(case):
    """The angle of each pair a position, and what the rotated elements are multiplied by."""
    theta = [BASE ** (-2.0 * i / case["dims"]) for i in range(case["dims"] // 2)]
    s = case["factor"]
    if case["scaling"] == "linear":
        return [x / s for x in theta], 1.0
    if case["scaling"] == "by_parts":
        share = [min(max((ORIGINAL * x / (2.0 * math.pi) - LOW) / (HIGH - LOW), 0.0), 1.0) for x in theta]
        return [x * (g + (1.0 - g) / s) for x, g in zip(theta, share)], 0.1 * math.log(s) + 1.0
    return theta, 1.0


def _prepare_rope(case, g):
    b, t, h, kvh, hd = (case[k] for k in ("batch", "tokens", "heads", "kv_heads", "head_dim"))
    dtype = TYPES[case["dtype"]]
    theta, magnitude = _frequencies(case)
    # every sequence begins somewhere; in a step each token stands alone
    start = (torch.rand((b, 1), generator=g, device=DEV) * max(1, case["furthest"] - t + 2)).long()
    s = {k: case[k] for k in ("op", "form", "batch", "tokens", "heads", "kv_heads", "head_dim", "dims", "pairs", "order")}
    s["positions"] = (start + torch.arange(t, device=DEV)).to(torch.int32)
    s["theta"] = torch.tensor(theta, dtype=torch.float64, device=DEV)
    s["magnitude"] = magnitude
    if case["form"] == "qkv" and case["op"] == "rope":
        s["qkv"] = _randn(g, b, t, (h + 2 * kvh) * hd).to(dtype)
    else:
        s["q"], s["k"] = _randn(g, b * h, t, hd).to(dtype), _randn(g, b * kvh, t, hd).to(dtype)
        s["v"] = _randn(g, b * kvh, t, hd).to(dtype) if case["form"] == "qkv" else None
    if own:
        from ff_input_projection_amd import Rope
        s["plan"] = Rope(b, t, h, hd, n_kv_heads=kvh, qkv_order=case["order"], pairs=case["pairs"],
                         rope_dims=case["dims"], rope_base=BASE, scaling=case["scaling"], factor=case["factor"],
                         original_tokens=ORIGINAL, low_turns=LOW, high_turns=HIGH, magnitude=magnitude, dtype=dtype)
    return s


def _prepare_attention(case, g):
    b, t, h, kvh, hd = (case[k] for k in ("batch", "tokens", "heads", "kv_heads", "head_dim"))
    # a few channels of the keys are far off, as rotated keys' slow channels are
    off = 2.0 * _randn(g, kvh, 1, hd) * (torch.rand((hd,), generator=g, device=DEV) < 0.06)
    q, k, v = _randn(g, b, h, t, hd), _randn(g, b, kvh, t, hd) + off, _randn(g, b, kvh, t, hd)
    if case["form"] == "qkv":
        # token-major, side by side, as one projection leaves them
        qkv = torch.cat([x.transpose(1, 2).reshape(b, t, -1) for x in (q, k, v)], -1).to(torch.bfloat16)
        q, k, v = (x.view(b, t, -1, hd).transpose(1, 2) for x in qkv.split([h * hd, kvh * hd, kvh * hd], -1))
    else:
        q, k, v = (x.to(torch.bfloat16).view(-1, t, hd) for x in (q, k, v))
    e = _extents(case)
    s = {"op": case["op"], "batch": b, "tokens": t, "heads": h, "kv_heads": kvh, "head_dim": hd, "q": q, "k": k, "v": v,
         "causal": case["causal"], "packed": case["sequences"] > 0,
         "extents": None if e is None else torch.tensor(e, dtype=torch.int32, device=DEV)}
    if case["op"] == "train":
        s["do"] = _randn(g, b, t, h * hd).to(torch.bfloat16)
    if own:
        from ff_input_projection_amd import PromptAttention
        s["plan"] = PromptAttention.for_tensors(q, k, v, batch=b, causal=case["causal"], sequences=case["sequences"])
        s["workspace"] = s["plan"].alloc_workspace(DEV)
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    return {"rope": _run_rope, "rope_grad": _run_rope_grad, "prompt": _run_prompt, "train": _run_train}[state["op"]](state)


def _columns(s):
    """[rows of q, k and v]: which heads of a token's row are q's, k's and v's."""
    h, kvh = s["heads"], s["kv_heads"]
    at = torch.arange(h + 2 * kvh, device=DEV)
    if s["order"] == "grouped":
        at = at.view(kvh, -1)
        return at[:, :h // kvh].flatten(), at[:, -2], at[:, -1]
    return at.split([h, kvh, kvh])


def _turn(s, x, back):
    """x [batch, tokens, heads, head_dim], rotated by its tokens' positions (or the transpose of that)."""
    phi = s["positions"].double()[:, :, None, None] * s["theta"]
    cos, sin = (phi.cos() * s["magnitude"]).float(), (phi.sin() * s["magnitude"]).float()
    if back:
        sin = -sin
    y, rest = x[..., :s["dims"]].float(), x[..., s["dims"]:].float()
    half = s["dims"] // 2
    a, b = (y[..., :half], y[..., half:]) if s["pairs"] == "half" else (y[..., 0::2], y[..., 1::2])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([a, b], -1) if s["pairs"] == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([y, rest], -1).to(x.dtype)


def _to_heads(x):
    """[batch, tokens, heads, head_dim] as [batch * heads, tokens, head_dim]."""
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])


def _from_heads(s, x):
    return x.view(s["batch"], -1, s["tokens"], s["head_dim"]).transpose(1, 2)


def _run_rope(s):
    if own:
        if s["form"] == "qkv":
            return s["plan"](s["qkv"], s["positions"])
        return s["plan"].rotate(s["q"], s["k"], s["positions"])
    if s["form"] == "heads":
        return tuple(_to_heads(_turn(s, _from_heads(s, s[n]), False)) for n in ("q", "k"))
    rows = s["qkv"].view(s["batch"], s["tokens"], -1, s["head_dim"])
    q, k, v = (rows[:, :, at] for at in _columns(s))
    return _to_heads(_turn(s, q, False)), _to_heads(_turn(s, k, False)), _to_heads(v)


def _run_rope_grad(s):
    if own:
        if s["form"] == "qkv":
            return s["plan"].backward(s["q"], s["k"], s["v"], s["positions"])
        return s["plan"].rotate_backward(s["q"], s["k"], s["positions"])
    q, k = (_turn(s, _from_heads(s, s[n]), True) for n in ("q", "k"))
    if s["form"] == "heads":
        return _to_heads(q), _to_heads(k)
    rows = torch.empty((s["batch"], s["tokens"], s["heads"] + 2 * s["kv_heads"], s["head_dim"]), dtype=q.dtype, device=DEV)
    for at, x in zip(_columns(s), (q, k, _from_heads(s, s["v"]))):
        rows[:, :, at] = x
    return rows.view(s["batch"], s["tokens"], -1)


def _by_group(s, x):
    """[batch, kv_heads, group * tokens, head_dim] in 32 bits."""
    return x.float().reshape(s["batch"], s["kv_heads"], -1, s["head_dim"])


def _seen(s):
    """[batch, 1, 1, tokens, tokens]: whether a row's token sees a column's."""
    at = torch.arange(s["tokens"], device=DEV)
    if s["packed"]:
        of = torch.searchsorted(s["extents"].long(), at, right=True)[None]
        real = (of > 0) & (of < s["extents"].numel())
        see = (of[:, :, None] == of[:, None, :]) & real[:, None, :]
    else:
        real = torch.ones((s["batch"], s["tokens"]), dtype=torch.bool, device=DEV)
        if s["extents"] is not None:
            real = at < s["extents"][:, None]
        see = real[:, None, :] & real[:, :, None]
    if s["causal"]:
        see = see & (at <= at[:, None])
    return see[:, None, None]


def _forward(s):
    """(o by groups in 32 bits, lse and probabilities [batch, kv_heads, group, tokens(, tokens)])."""
    t = s["tokens"]
    q, k, v = (_by_group(s, s[n]) for n in ("q", "k", "v"))
    x = (q @ k.transpose(-1, -2)).view(s["batch"], s["kv_heads"], -1, t, t) * s["head_dim"] ** -0.5
    x = x.masked_fill(~_seen(s), -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    return p.flatten(2, 3) @ v, (top + total.log()).squeeze(-1), p


def _tokens_major(s, o):
    return o.view(s["batch"], s["heads"], s["tokens"], -1).transpose(1, 2).reshape(s["batch"], s["tokens"], -1).to(torch.bfloat16)


def _run_prompt(s):
    if own:
        return s["plan"](s["q"], s["k"], s["v"], s["extents"])
    o, lse, _ = _forward(s)
    return _tokens_major(s, o), lse.reshape(-1, s["tokens"])


def _run_train(s):
    if own:
        o, lse = s["plan"](s["q"], s["k"], s["v"], s["extents"])
        return o, lse, *s["plan"].backward(s["q"], s["k"], s["v"], o, lse, s["do"], s["extents"], workspace=s["workspace"])
    o, lse, p = _forward(s)
    q, k, v = (_by_group(s, s[n]) for n in ("q", "k", "v"))
    do = _by_group(s, s["do"].view(s["batch"], s["tokens"], s["heads"], -1).transpose(1, 2))
    dp = (do @ v.transpose(-1, -2)).view(p.shape)
    ds = p * (dp - (do * o).sum(-1).view(p.shape[:-1])[..., None])
    p, ds = p.flatten(2, 3), ds.flatten(2, 3) * s["head_dim"] ** -0.5
    grads = ds @ k, ds.transpose(-1, -2) @ q, p.transpose(-1, -2) @ do
    return _tokens_major(s, o), lse.reshape(-1, s["tokens"]), *(x.reshape(s[n].shape).to(torch.bfloat16) for n, x in zip("qkv", grads))


# ------------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    b, t, h, kvh, hd = (case[k] for k in ("batch", "tokens", "heads", "kv_heads", "head_dim"))
    if case["op"] in ("rope", "rope_grad"):
        size = 2 if case["dtype"] == "bf16" else 4
        moved = h + 2 * kvh if case["form"] == "qkv" else h + kvh
        return {"bytes": 2 * b * t * moved * hd * size + 4 * b * t, "flops": 3 * b * t * (h + kvh) * case["dims"]}
    pairs = sum((y - x) * (y - x + 1) // 2 if case["causal"] else (y - x) ** 2 for _, x, y in _spans(case))
    q, kv = b * t * h * hd * 2, 2 * b * t * kvh * hd * 2
    bytes_, flops = 2 * q + kv + 4 * b * t * h, 4 * pairs * h * hd
    if case["op"] == "train":
        bytes_, flops = bytes_ + 4 * q + 2 * kv + 4 * b * t * h, flops + 10 * pairs * h * hd
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_rope if case["op"] in ("rope", "rope_grad") else _exact_attention)(case, s)


def _exact_turn(case, s, x, back):
    """Pairs as complex numbers, times magnitude e^(i p theta)."""
    theta, magnitude = _frequencies(case)
    z = torch.polar(torch.full((1,), magnitude, dtype=torch.float64, device=DEV),
                    s["positions"].double()[..., None] * torch.tensor(theta, dtype=torch.float64, device=DEV))
    if back:
        z = z.conj()
    y = x.double().clone()
    n = case["dims"]
    first, second = (slice(0, n // 2), slice(n // 2, n)) if case["pairs"] == "half" else (slice(0, n, 2), slice(1, n, 2))
    w = torch.complex(y[..., first], y[..., second]) * z[:, None]
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _exact_rope(case, s):
    b, t, h, kvh, hd = (case[k] for k in ("batch", "tokens", "heads", "kv_heads", "head_dim"))
    group = h // kvh
    if case["op"] == "rope" and case["form"] == "qkv":
        x = s["qkv"].double().view(b, t, -1, hd).permute(0, 2, 1, 3)
        if case["order"] == "grouped":
            x = x.reshape(b, kvh, group + 2, t, hd)
            q, k, v = x[:, :, :group].reshape(b, h, t, hd), x[:, :, group], x[:, :, group + 1]
        else:
            q, k, v = x[:, :h], x[:, h:h + kvh], x[:, h + kvh:]
        return tuple(x.reshape(-1, t, hd) for x in (_exact_turn(case, s, q, False), _exact_turn(case, s, k, False), v))
    q, k = (_exact_turn(case, s, s[n].view(b, -1, t, hd), case["op"] == "rope_grad") for n in ("q", "k"))
    if case["form"] == "heads":
        return q.reshape(-1, t, hd), k.reshape(-1, t, hd)
    v = s["v"].double().view(b, kvh, t, hd)
    if case["order"] == "grouped":
        x = torch.cat([q.view(b, kvh, group, t, hd), k[:, :, None], v[:, :, None]], 2).reshape(b, -1, t, hd)
    else:
        x = torch.cat([q, k, v], 1)
    return x.permute(0, 2, 1, 3).reshape(b, t, -1)


def _exact_attention(case, s):
    b, t, h, kvh, hd = (case[k] for k in ("batch", "tokens", "heads", "kv_heads", "head_dim"))
    group, train = h // kvh, case["op"] == "train"
    whole = dict(dtype=torch.float64, device=DEV)
    q, k, v = (s[n].reshape(b, -1, t, hd) for n in ("q", "k", "v"))
    o, lse = torch.zeros((b, t, h, hd), **whole), torch.full((b, h, t), -math.inf, **whole)
    dq, dk, dv = (torch.zeros(x.shape, **whole) for x in (q, k, v))
    for row, x0, x1 in _spans(case):
        if x0 == x1:
            continue
        late = torch.ones((x1 - x0, x1 - x0), dtype=torch.bool, device=DEV).triu(1) if case["causal"] else None
        for i in range(h):
            a, c, d = q[row, i, x0:x1].double(), k[row, i // group, x0:x1].double(), v[row, i // group, x0:x1].double()
            x = torch.mm(a, c.t().contiguous()) / math.sqrt(hd)
            if late is not None:
                x.masked_fill_(late, -math.inf)
            lse[row, i, x0:x1] = x.logsumexp(-1)
            x = x.softmax(-1)
            y = torch.mm(x, d)
            o[row, x0:x1, i] = y
            if train:
                do = s["do"].view(b, t, h, hd)[row, x0:x1, i].double()
                dv[row, i // group, x0:x1] += torch.mm(x.t(), do)
                x = x * torch.mm(do, d.t()) - x * (do * y).sum(-1, keepdim=True)
                dq[row, i, x0:x1] = torch.mm(x, c) / math.sqrt(hd)
                dk[row, i // group, x0:x1] += torch.mm(x.t(), a) / math.sqrt(hd)
    o, lse = o.view(b, t, h * hd), lse.view(b * h, t)
    return (o, lse, dq.view(s["q"].shape), dk.view(s["k"].shape), dv.view(s["v"].shape)) if train else (o, lse)
