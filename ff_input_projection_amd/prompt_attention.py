"""Attention over whole prompts, forward and backward (binding of ``include/prompt_attention.h``)."""
from __future__ import annotations

import ctypes

import torch

from . import OK, FusedProjError, PromptAttentionDesc, _DTYPES, _planned_call, _planned_call_function, load_library
from .layer_norm import _allocate_on


def make_prompt_attention_desc(batch: int, tokens: int, n_heads: int, head_dim: int, *, n_kv_heads: int = 0,
                               causal: bool = True, sequences: int = 0, sm_scale: float = 0.0, q_strides=None,
                               k_strides=None, v_strides=None, dtype: torch.dtype = torch.bfloat16) -> PromptAttentionDesc:
    """Strides: elements between batch rows, heads and tokens; None for head-major and dense."""
    d = PromptAttentionDesc()
    d.dtype, d.causal = _DTYPES[dtype], int(bool(causal))
    d.batch, d.tokens, d.n_heads, d.n_kv_heads, d.head_dim = batch, tokens, n_heads, n_kv_heads, head_dim
    d.sequences, d.sm_scale = sequences, float(sm_scale)
    kvh = n_kv_heads if n_kv_heads > 0 else n_heads
    for to, strides, heads in ((d.q_strides, q_strides, n_heads), (d.k_strides, k_strides, kvh), (d.v_strides, v_strides, kvh)):
        to[:] = tuple(strides) if strides is not None else (heads * tokens * head_dim, tokens * head_dim, head_dim)
    return d


def validate_prompt_attention(desc: PromptAttentionDesc) -> int:
    return load_library().prompt_attention_validate(ctypes.byref(desc))


class PromptAttention:
    """One planned attention of whole sequences over themselves (see prompt_attention.h).

    ``sequences`` = 0: a padded batch, ``extents`` [b] int32 its lengths (None: all T tokens);
    ``sequences`` = n: packed, batch 1, ``extents`` [n + 1] int32 the offsets. Call with q
    [b*H, T, hd], k and v [b*KVH, T, hd] (what a projection gives; with strides in the plan, or made by
    ``for_tensors``, 4-dimensional views [b, heads, T, hd]); returns ``(o, lse)``: o [b, T, H*hd], lse
    fp32 [b*H, T]. ``backward(q, k, v, o, lse, do, extents)`` returns ``(dq, dk, dv)``, dense and
    shaped like q, k and v. Outputs may be passed in; launches go to torch's current stream (or
    ``stream``) and are asynchronous. A plan belongs to the device that was current when it was
    made: its tensors are on that device, and it is the current one in every call.
    """

    def __init__(self, batch: int, tokens: int, n_heads: int, head_dim: int, **kw):
        self._lib = load_library()
        self.desc = d = make_prompt_attention_desc(batch, tokens, n_heads, head_dim, **kw)
        self.B, self.T, self.H, self.hd, self.sequences = batch, tokens, n_heads, head_dim, d.sequences
        self.KVH = d.n_kv_heads if d.n_kv_heads > 0 else n_heads
        h = ctypes.c_void_p()
        rc = self._lib.prompt_attention_create(ctypes.byref(d), ctypes.byref(h))
        if rc != OK:
            raise FusedProjError(rc, "prompt_attention_create")
        self._h, self._device = h, torch.cuda.current_device()
        n = ctypes.c_size_t()
        rc = self._lib.prompt_attention_backward_workspace_size(h, ctypes.byref(n))
        if rc != OK:
            raise FusedProjError(rc, "prompt_attention_backward_workspace_size")
        self._workspace_bytes = int(n.value)
        # [b*heads, T, hd], or [b, heads, T, hd] where a tensor has strides of its own
        self._shapes, self._strides = [], []
        for name, heads in (("q_strides", self.H), ("k_strides", self.KVH), ("v_strides", self.KVH)):
            if kw.get(name) is None:
                self._shapes.append((batch * heads, tokens, head_dim))
                self._strides.append(None)
            else:
                self._shapes.append((batch, heads, tokens, head_dim))
                self._strides.append((*kw[name], 1))
        self._o_shape, self._lse_shape = (batch, tokens, n_heads * head_dim), (batch * n_heads, tokens)
        self._extents_shape = (self.sequences + 1,) if self.sequences else (batch,)
        # the usual calls (outputs allocated, the current stream) in one step; whatever they do not
        # take goes through the checks below
        bf16, f32 = torch.bfloat16, torch.float32
        qkv = tuple(("in", s, t, bf16) for s, t in zip(self._shapes, self._strides))
        extents = ("maybe", self._extents_shape, None, torch.int32)
        self._forward = _planned_call("prompt_attention_run", h, (*qkv, extents, ("out", self._o_shape, bf16),
                                                                  ("out", self._lse_shape, f32)))
        self._backward = _planned_call(
            "prompt_attention_backward", h,
            (*qkv, extents, ("in", self._o_shape, None, bf16), ("in", self._lse_shape, None, f32),
             ("in", self._o_shape, None, bf16), *(("out", s, bf16) for s in self._shapes), ("workspace", self._workspace_bytes)))
        self._call = _planned_call_function()

    @classmethod
    def for_tensors(cls, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, batch: int = 1, **kw) -> "PromptAttention":
        """A plan for tensors like these: views [b, heads, T, hd] of any strides, or (all three) [b*heads, T, hd] with
        ``batch`` rows."""
        if q.dim() == 3:
            if k.dim() != 3 or v.dim() != 3 or batch < 1 or q.shape[0] % batch or k.shape[0] % batch:
                raise ValueError(f"q, k and v have shapes {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)} for a batch of {batch}")
            return cls(batch, q.shape[1], q.shape[0] // batch, q.shape[2], n_kv_heads=k.shape[0] // batch, dtype=q.dtype, **kw)
        if q.dim() != 4 or k.dim() != 4 or v.dim() != 4 or any(t.stride(3) != 1 for t in (q, k, v)):
            raise ValueError("q, k and v are [b, heads, T, hd] with neighbouring elements, or [b*heads, T, hd]")
        return cls(q.shape[0], q.shape[2], q.shape[1], q.shape[3], n_kv_heads=k.shape[1], q_strides=q.stride()[:3],
                   k_strides=k.stride()[:3], v_strides=v.stride()[:3], dtype=q.dtype, **kw)

    def workspace_bytes(self) -> int:
        """Device workspace the backward pass needs."""
        return self._workspace_bytes

    def alloc_workspace(self, device) -> torch.Tensor:
        return torch.empty((self.workspace_bytes(),), dtype=torch.uint8, device=device)

    def _check(self, name, t, shape, device, dtype=torch.bfloat16, strides=None):
        fits = t is not None and t.shape == shape and t.dtype == dtype and t.device == device
        if not fits or (not t.is_contiguous() if strides is None else t.stride() != strides):
            how = "a contiguous" if strides is None else f"a (strides {strides})"
            raise ValueError(f"{name} must be {how} {tuple(shape)} {dtype} tensor on {device}")

    def _check_inputs(self, q, k, v, extents):
        dev = q.device
        if dev.type != "cuda":
            raise TypeError("q, k and v are GPU tensors")
        if dev.index != self._device:
            raise ValueError(f"the plan is for cuda:{self._device}, not for {dev}")
        for name, t, shape, strides in zip(("q", "k", "v"), (q, k, v), self._shapes, self._strides):
            self._check(name, t, shape, dev, strides=strides)
        if extents is not None:
            self._check("extents", extents, self._extents_shape, dev, torch.int32)
        elif self.sequences:
            raise ValueError("packed sequences need their offsets")
        return dev

    def __call__(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, extents: torch.Tensor | None = None, out=None,
                 stream: torch.cuda.Stream | None = None):
        if out is None and stream is None and self._forward is not None and (extents is not None or not self.sequences):
            r = self._call(self._forward, q, k, v, extents, None)
            if type(r) is tuple:
                return r
            if r is not None:
                raise FusedProjError(r, "prompt_attention_run")
        dev = self._check_inputs(q, k, v, extents)
        if out is None:
            with _allocate_on(stream):
                out = (torch.empty(self._o_shape, dtype=torch.bfloat16, device=dev),
                       torch.empty(self._lse_shape, dtype=torch.float32, device=dev))
        o, lse = out
        self._check("o", o, self._o_shape, dev)
        if lse is not None:
            self._check("lse", lse, self._lse_shape, dev, torch.float32)
        st = stream if stream is not None else torch.cuda.current_stream(dev)
        rc = self._lib.prompt_attention_run(self._h, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                            None if extents is None else extents.data_ptr(), o.data_ptr(),
                                            None if lse is None else lse.data_ptr(), st.cuda_stream)
        if rc != OK:
            raise FusedProjError(rc, "prompt_attention_run")
        return o, lse

    def backward(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor, do: torch.Tensor,
                 extents: torch.Tensor | None = None, out=None, workspace: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None):
        """Gradients (dq, dk, dv) for the upstream gradient ``do`` [b, T, H*hd] and the forward pass's o and lse."""
        if out is None and stream is None and self._backward is not None and (extents is not None or not self.sequences):
            r = self._call(self._backward, q, k, v, extents, o, lse, do, workspace)
            if type(r) is tuple:
                return r
            if r is not None:
                raise FusedProjError(r, "prompt_attention_backward")
        dev = self._check_inputs(q, k, v, extents)
        self._check("o", o, self._o_shape, dev)
        self._check("lse", lse, self._lse_shape, dev, torch.float32)
        self._check("do", do, self._o_shape, dev)
        with _allocate_on(stream):
            if out is None:
                out = tuple(torch.empty(s, dtype=torch.bfloat16, device=dev) for s in self._shapes)
            if workspace is None:
                workspace = torch.empty((self._workspace_bytes,), dtype=torch.uint8, device=dev)
        dq, dk, dv = out
        for name, t, shape in zip(("dq", "dk", "dv"), (dq, dk, dv), self._shapes):
            self._check(name, t, shape, dev)
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        st = stream if stream is not None else torch.cuda.current_stream(dev)
        rc = self._lib.prompt_attention_backward(self._h, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                                 None if extents is None else extents.data_ptr(), o.data_ptr(),
                                                 lse.data_ptr(), do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                                 workspace.data_ptr(), workspace.numel() * workspace.element_size(), st.cuda_stream)
        if rc != OK:
            raise FusedProjError(rc, "prompt_attention_backward")
        return dq, dk, dv

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._forward = self._backward = None
            self._lib.prompt_attention_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
