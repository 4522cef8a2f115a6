"""Layer norm of the activation that a fused projection reads (binding of ``include/layer_norm.h``)."""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import OK, FusedProjError, LayerNormDesc, _DTYPES, _fill_activation, _planned_call, _planned_call_function, load_library


def make_layer_norm_desc(x_shape, x_strides, layout: str, dtype: torch.dtype, *, eps: float = 1e-5,
                         has_bias: bool = True) -> LayerNormDesc:
    """Descriptor from an activation's shape and element strides (layouts as for make_desc)."""
    d = LayerNormDesc()
    d.dtype = _DTYPES[dtype]
    if layout == "channels_first" and not 3 <= len(x_shape) <= 5 or layout == "tokens_last" and len(x_shape) != 3:
        raise ValueError(f"x of shape {tuple(x_shape)} is not {layout}")
    _fill_activation(d, tuple(x_shape), tuple(x_strides), layout)
    d.has_bias, d.eps = int(bool(has_bias)), float(eps)
    return d


def validate_layer_norm(desc: LayerNormDesc) -> int:
    return load_library().layer_norm_validate(ctypes.byref(desc))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _allocate_on(stream):
    """Memory that a call allocates belongs to the stream that the call's kernels run on."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class LayerNorm:
    """One planned layer norm over the channels of an activation (see layer_norm.h).

    Call with device tensors ``x`` (shape, strides and dtype as planned), ``gamma`` [C] and,
    with a bias, ``beta`` [C]; returns ``(y, stats)``: y dense in x's shape, stats fp32
    [2, b*S] with every token's mean and 1 / standard deviation (what ``backward`` takes).
    ``backward`` returns ``(dx, dgamma, dbeta)``, dbeta None without a bias. Outputs may be
    passed in; the launches go to torch's current stream (or ``stream``) and are asynchronous.
    A plan belongs to the device that was current when it was made: its tensors are on that
    device, and it is the current one in every call.
    """

    def __init__(self, x_shape, x_strides, layout: str, dtype: torch.dtype, *, eps: float = 1e-5, has_bias: bool = True):
        self._lib = load_library()
        self.desc = make_layer_norm_desc(x_shape, x_strides, layout, dtype, eps=eps, has_bias=has_bias)
        self.x_shape, self.x_strides, self.layout, self.dtype = tuple(x_shape), tuple(x_strides), layout, dtype
        self.has_bias, self.C = bool(has_bias), int(self.desc.channels)
        self.M = int(self.desc.batch)
        for i in range(self.desc.n_spatial):
            self.M *= int(self.desc.spatial[i])
        h = ctypes.c_void_p()
        rc = self._lib.layer_norm_create(ctypes.byref(self.desc), ctypes.byref(h))
        if rc != OK:
            raise FusedProjError(rc, "layer_norm_create")
        self._h, self._device = h, torch.cuda.current_device()
        n = ctypes.c_size_t()
        rc = self._lib.layer_norm_backward_workspace_size(self._h, ctypes.byref(n))
        if rc != OK:
            raise FusedProjError(rc, "layer_norm_backward_workspace_size")
        self._workspace_bytes = int(n.value)
        # the usual call (outputs allocated, the current stream) in one step; whatever it does not
        # take goes through the checks below
        x, c, stats = ("in", self.x_shape, self.x_strides, dtype), ("in", (self.C,), None, dtype), (2, self.M)
        beta = c if self.has_bias else ("maybe", (self.C,), None, dtype)
        self._forward = _planned_call("layer_norm_run", h, (x, c, beta, ("out", self.x_shape, dtype),
                                                            ("out", stats, torch.float32)))
        self._backward = None
        if self.has_bias:
            self._backward = _planned_call(
                "layer_norm_backward", h,
                (x, c, ("in", stats, None, torch.float32), ("in", self.x_shape, None, dtype), ("out", self.x_shape, dtype),
                 ("out", (self.C,), dtype), ("out", (self.C,), dtype), ("workspace", self._workspace_bytes)))
        self._call = _planned_call_function()

    @classmethod
    def for_tensor(cls, x: torch.Tensor, layout: str, **kw) -> "LayerNorm":
        return cls(x.shape, x.stride(), layout, x.dtype, **kw)

    def workspace_bytes(self) -> int:
        """Device workspace the backward pass needs."""
        return self._workspace_bytes

    def _check_x(self, x):
        if x.shape != self.x_shape or x.stride() != self.x_strides:
            raise ValueError(f"x has shape {tuple(x.shape)} strides {x.stride()}; planned for {self.x_shape} / "
                             f"{self.x_strides}")
        if x.dtype != self.dtype or not x.is_cuda:
            raise TypeError(f"x must be a {self.dtype} GPU tensor")
        if x.device.index != self._device:
            raise ValueError(f"the plan is for cuda:{self._device}, not for {x.device}")

    def _check(self, name, t, shape, device, dtype=None):
        if t is None or t.shape != shape or not t.is_contiguous() or t.dtype != (dtype or self.dtype) or t.device != device:
            raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype or self.dtype} tensor on {device}")

    def __call__(self, x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor | None = None, out=None,
                 stream: torch.cuda.Stream | None = None):
        if out is None and stream is None and self._forward is not None:
            r = self._call(self._forward, x, gamma, beta if self.has_bias else None, None)
            if type(r) is tuple:
                return r
            if r is not None:
                raise FusedProjError(r, "layer_norm_run")
        self._check_x(x)
        dev = x.device
        self._check("gamma", gamma, (self.C,), dev)
        if self.has_bias:
            self._check("beta", beta, (self.C,), dev)
        if out is None:
            with _allocate_on(stream):
                y = torch.empty(self.x_shape, dtype=self.dtype, device=dev)
                stats = torch.empty((2, self.M), dtype=torch.float32, device=dev)
        else:
            y, stats = out
            self._check("y", y, self.x_shape, dev)
            if stats is not None:
                self._check("stats", stats, (2, self.M), dev, torch.float32)
        st = stream if stream is not None else torch.cuda.current_stream(dev)
        rc = self._lib.layer_norm_run(self._h, x.data_ptr(), gamma.data_ptr(), beta.data_ptr() if self.has_bias else None,
                                      y.data_ptr(), _ptr(stats), st.cuda_stream)
        if rc != OK:
            raise FusedProjError(rc, "layer_norm_run")
        return y, stats

    def backward(self, x: torch.Tensor, gamma: torch.Tensor, stats: torch.Tensor, dy: torch.Tensor, out=None,
                 workspace: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
        """Gradients (dx, dgamma, dbeta) for the upstream gradient ``dy`` (dense, shaped like x) and
        the forward pass's ``stats``. The workspace (uint8 device tensor of at least
        workspace_bytes()) is allocated when not given."""
        if out is None and stream is None and self._backward is not None:
            r = self._call(self._backward, x, gamma, stats, dy, workspace)
            if type(r) is tuple:
                return r
            if r is not None:
                raise FusedProjError(r, "layer_norm_backward")
        self._check_x(x)
        dev = x.device
        self._check("gamma", gamma, (self.C,), dev)
        self._check("stats", stats, (2, self.M), dev, torch.float32)
        self._check("dy", dy, self.x_shape, dev)
        with _allocate_on(stream):
            if out is None:
                dx = torch.empty(self.x_shape, dtype=self.dtype, device=dev)
                dgamma = torch.empty((self.C,), dtype=self.dtype, device=dev)
                dbeta = torch.empty((self.C,), dtype=self.dtype, device=dev) if self.has_bias else None
            if workspace is None:
                workspace = torch.empty((self._workspace_bytes,), dtype=torch.uint8, device=dev)
        if out is not None:
            dx, dgamma, dbeta = out
            self._check("dx", dx, self.x_shape, dev)
            self._check("dgamma", dgamma, (self.C,), dev)
            if self.has_bias:
                self._check("dbeta", dbeta, (self.C,), dev)
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        st = stream if stream is not None else torch.cuda.current_stream(dev)
        rc = self._lib.layer_norm_backward(self._h, x.data_ptr(), gamma.data_ptr(), stats.data_ptr(), dy.data_ptr(),
                                           dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr() if self.has_bias else None,
                                           workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                           st.cuda_stream)
        if rc != OK:
            raise FusedProjError(rc, "layer_norm_backward")
        return dx, dgamma, dbeta if self.has_bias else None

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._forward = self._backward = None
            self._lib.layer_norm_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
