"""Rotary positions, every token at a position of its own (binding of ``include/rope.h``)."""
from __future__ import annotations

import ctypes

import torch

from . import (OK, QKV_CONTIGUOUS, QKV_GROUPED, FusedProjError, RopeDesc, _DTYPES, _planned_call, _planned_call_function,
               load_library)
from .layer_norm import _allocate_on

PAIRS = {"half": 0, "interleaved": 1}
SCALINGS = {"none": 0, "linear": 1, "by_parts": 2}


def make_rope_desc(batch: int, tokens: int, n_heads: int, head_dim: int, *, n_kv_heads: int = 0,
                   qkv_order: str = "contiguous", rope_dims: int = 0, pairs: str = "half", rope_base: float = 10000.0,
                   scaling: str = "none", factor: float = 1.0, original_tokens: int = 1, low_turns: float = 1.0,
                   high_turns: float = 32.0, magnitude: float = 1.0, dtype: torch.dtype = torch.bfloat16) -> RopeDesc:
    d = RopeDesc()
    d.dtype = _DTYPES[dtype]
    d.qkv_order = {"contiguous": QKV_CONTIGUOUS, "grouped": QKV_GROUPED}[qkv_order]
    d.batch, d.tokens, d.n_heads, d.n_kv_heads, d.head_dim = batch, tokens, n_heads, n_kv_heads, head_dim
    d.rope_dims, d.pairs, d.scaling = rope_dims, PAIRS[pairs], SCALINGS[scaling]
    d.rope_base, d.factor, d.original_tokens = float(rope_base), float(factor), original_tokens
    d.low_turns, d.high_turns, d.magnitude = float(low_turns), float(high_turns), float(magnitude)
    return d


def validate_rope(desc: RopeDesc) -> int:
    return load_library().rope_validate(ctypes.byref(desc))


class Rope:
    """One planned rotation by positions (see rope.h): halves or neighbours paired, the whole head
    or its first ``rope_dims`` elements, frequencies scaled for long contexts ("linear", or
    "by_parts" with ``original_tokens``, ``low_turns``, ``high_turns`` and ``magnitude``).

    Call with ``qkv`` [b, T, (H + 2*KVH)*hd] and ``positions`` [b, T] int32 (None: 0 .. T - 1 in
    every sequence); returns ``(q, k, v)`` [b*H or b*KVH, T, hd] with q and k rotated, and
    ``backward(dq, dk, dv, positions)`` returns dqkv. ``rotate(q, k, positions)`` rotates
    head-major q and k, in place with ``out=(q, k)``; ``rotate_backward(dq, dk, positions)`` is
    its backward pass. Outputs may be passed in; launches go to torch's current stream (or
    ``stream``) and are asynchronous. A plan belongs to the device that was current when it was
    made: its tensors are on that device, and it is the current one in every call. It holds the pairs'
    angles in device memory, so keep it as long as a graph that captured its calls is replayed.
    """

    def __init__(self, batch: int, tokens: int, n_heads: int, head_dim: int, **kw):
        self._lib = load_library()
        self.desc = d = make_rope_desc(batch, tokens, n_heads, head_dim, **kw)
        self.dtype = kw.get("dtype", torch.bfloat16)
        self.B, self.T, self.H, self.hd = batch, tokens, n_heads, head_dim
        self.KVH = d.n_kv_heads if d.n_kv_heads > 0 else n_heads
        h = ctypes.c_void_p()
        rc = self._lib.rope_create(ctypes.byref(d), ctypes.byref(h))
        if rc != OK:
            raise FusedProjError(rc, "rope_create")
        self._h, self._device = h, torch.cuda.current_device()
        self._rows_shape, self._q_shape, self._kv_shape = self.shapes()
        # the usual calls (outputs allocated, the current stream) in one step; whatever they do not
        # take goes through the checks below
        slot = lambda kind, shape: (kind, shape, None, self.dtype) if kind == "in" else (kind, shape, self.dtype)
        at = ("maybe", (batch, tokens), None, torch.int32)
        rows, q, kv = ((slot("in", s), slot("out", s)) for s in (self._rows_shape, self._q_shape, self._kv_shape))
        self._split = _planned_call("rope_split", h, (rows[0], at, q[1], kv[1], kv[1]))
        self._split_backward = _planned_call("rope_split_backward", h, (q[0], kv[0], kv[0], at, rows[1]))
        self._rotate = _planned_call("rope_rotate", h, (q[0], kv[0], at, q[1], kv[1]))
        self._rotate_backward = _planned_call("rope_rotate_backward", h, (q[0], kv[0], at, q[1], kv[1]))
        self._call = _planned_call_function()

    def shapes(self):
        """Shapes of qkv, of q, and of k and v."""
        return ((self.B, self.T, (self.H + 2 * self.KVH) * self.hd), (self.B * self.H, self.T, self.hd),
                (self.B * self.KVH, self.T, self.hd))

    def _check(self, name, t, shape, device, dtype=None):
        if t is None or t.shape != shape or not t.is_contiguous() or t.dtype != (dtype or self.dtype) or t.device != device:
            raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype or self.dtype} tensor on {device}")

    def _run(self, function, inputs, positions, shapes, out, stream):
        """Checks, allocates and calls: inputs {name: (tensor, shape)}, shapes of the outputs."""
        dev = next(iter(inputs.values()))[0].device
        if dev.type != "cuda":
            raise TypeError("the tensors of a rotation are GPU tensors")
        if dev.index != self._device:
            raise ValueError(f"the plan is for cuda:{self._device}, not for {dev}")
        for name, (t, shape) in inputs.items():
            self._check(name, t, shape, dev)
        if positions is not None:
            self._check("positions", positions, (self.B, self.T), dev, torch.int32)
        if out is None:
            with _allocate_on(stream):
                out = tuple(torch.empty(s, dtype=self.dtype, device=dev) for s in shapes)
        if len(out) != len(shapes):
            raise ValueError(f"{len(out)} outputs are given, {len(shapes)} are wanted")
        for t, shape in zip(out, shapes):
            self._check("an output", t, shape, dev)
        st = stream if stream is not None else torch.cuda.current_stream(dev)
        at = None if positions is None else positions.data_ptr()
        rc = getattr(self._lib, function)(self._h, *(t.data_ptr() for t, _ in inputs.values()), at,
                                          *(t.data_ptr() for t in out), st.cuda_stream)
        if rc != OK:
            raise FusedProjError(rc, function)
        return tuple(out)

    def __call__(self, qkv: torch.Tensor, positions: torch.Tensor | None = None, out=None,
                 stream: torch.cuda.Stream | None = None):
        if out is None and stream is None and self._split is not None:
            r = self._call(self._split, qkv, positions, None)
            if type(r) is tuple:
                return r
            if r is not None:
                raise FusedProjError(r, "rope_split")
        return self._run("rope_split", {"qkv": (qkv, self._rows_shape)}, positions,
                         (self._q_shape, self._kv_shape, self._kv_shape), out, stream)

    def backward(self, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor, positions: torch.Tensor | None = None,
                 out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
        """The gradient of qkv from those of q, k and v."""
        if out is None and stream is None and self._split_backward is not None:
            r = self._call(self._split_backward, dq, dk, dv, positions, None)
            if type(r) is tuple:
                return r[0]
            if r is not None:
                raise FusedProjError(r, "rope_split_backward")
        inputs = {"dq": (dq, self._q_shape), "dk": (dk, self._kv_shape), "dv": (dv, self._kv_shape)}
        return self._run("rope_split_backward", inputs, positions, (self._rows_shape,), None if out is None else (out,),
                         stream)[0]

    def rotate(self, q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor | None = None, out=None,
               stream: torch.cuda.Stream | None = None):
        if out is None and stream is None and self._rotate is not None:
            r = self._call(self._rotate, q, k, positions, None)
            if type(r) is tuple:
                return r
            if r is not None:
                raise FusedProjError(r, "rope_rotate")
        return self._run("rope_rotate", {"q": (q, self._q_shape), "k": (k, self._kv_shape)}, positions,
                         (self._q_shape, self._kv_shape), out, stream)

    def rotate_backward(self, dq: torch.Tensor, dk: torch.Tensor, positions: torch.Tensor | None = None, out=None,
                        stream: torch.cuda.Stream | None = None):
        """The gradients of what ``rotate`` took, from those of what it gave."""
        if out is None and stream is None and self._rotate_backward is not None:
            r = self._call(self._rotate_backward, dq, dk, positions, None)
            if type(r) is tuple:
                return r
            if r is not None:
                raise FusedProjError(r, "rope_rotate_backward")
        return self._run("rope_rotate_backward", {"dq": (dq, self._q_shape), "dk": (dk, self._kv_shape)}, positions,
                         (self._q_shape, self._kv_shape), out, stream)

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._split = self._split_backward = self._rotate = self._rotate_backward = None
            self._lib.rope_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
