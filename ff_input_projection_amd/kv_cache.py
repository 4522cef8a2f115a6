"""Key/value cache in 4 or 8 bits and the attention over it (binding of ``include/kv_cache.h``)."""
from __future__ import annotations

import ctypes

import torch

from . import OK, FusedProjError, KVCacheDesc, KVCacheStorage, _DTYPES, _planned_call, _planned_call_function, load_library
from .layer_norm import _allocate_on


def make_kv_cache_desc(batch: int, tokens: int, n_heads: int, head_dim: int, *, n_kv_heads: int = 0, bits: int = 4,
                       page_size: int = 64, n_pages: int, max_pages: int, sm_scale: float = 0.0,
                       dtype: torch.dtype = torch.bfloat16) -> KVCacheDesc:
    d = KVCacheDesc()
    d.dtype, d.bits = _DTYPES[dtype], bits
    d.batch, d.tokens, d.n_heads, d.n_kv_heads, d.head_dim = batch, tokens, n_heads, n_kv_heads, head_dim
    d.page_size, d.n_pages, d.max_pages, d.sm_scale = page_size, n_pages, max_pages, float(sm_scale)
    return d


def validate_kv_cache(desc: KVCacheDesc) -> int:
    return load_library().kv_cache_validate(ctypes.byref(desc))


class KVCache:
    """One planned step over a paged, quantised k/v cache (see kv_cache.h): up to ``tokens``
    tokens in each of ``batch`` sequences.

    The cache's memory is the caller's: ``alloc_storage(device)`` makes it once, and every plan
    with the same k/v heads, head size, bits and pages uses it (a plan for prompts and one for
    single tokens, say). ``table`` [batch, max_pages], ``lengths`` [batch] and ``counts``
    [batch] (None: ``tokens`` each) are int32 GPU tensors: the pages of a sequence, the tokens
    that the cache holds of it after the step, and how many of them are the step's own (the
    last ones; the rest of the ``tokens`` is padding).

    ``write(storage, k, v, ...)`` quantises k and v [batch*KVH, tokens, hd] into their slots;
    ``read`` returns the step's rows as the values they stand for; ``attend`` returns
    [batch, tokens, H*hd], the step's queries q [batch*H, tokens, hd] over all that the cache
    holds up to each. Launches go to torch's current stream (or ``stream``) and are
    asynchronous. A plan belongs to the device that was current when it was made: its tensors
    are on that device, and it is the current one in every call.
    """

    def __init__(self, batch: int, tokens: int, n_heads: int, head_dim: int, **kw):
        self._lib = load_library()
        self.desc = d = make_kv_cache_desc(batch, tokens, n_heads, head_dim, **kw)
        self.B, self.T, self.H, self.hd, self.bits = batch, tokens, n_heads, head_dim, d.bits
        self.KVH = d.n_kv_heads if d.n_kv_heads > 0 else n_heads
        h = ctypes.c_void_p()
        rc = self._lib.kv_cache_create(ctypes.byref(d), ctypes.byref(h))
        if rc != OK:
            raise FusedProjError(rc, "kv_cache_create")
        self._h, self._device = h, torch.cuda.current_device()
        self._table_shape, self._kv_shape = (batch, d.max_pages), (batch * self.KVH, tokens, head_dim)
        self._q_shape, self._o_shape = (batch * n_heads, tokens, head_dim), (batch, tokens, n_heads * head_dim)
        slots = (d.n_pages, self.KVH, d.page_size)
        self._codes_shape, self._params_shape = slots + (head_dim * d.bits // 8,), slots + (2,)
        n = ctypes.c_size_t()
        rc = self._lib.kv_cache_attend_workspace_size(self._h, ctypes.byref(n))
        self._workspace_bytes = int(n.value) if rc == OK else None   # None: a head size attention does not take
        # the usual calls (outputs allocated, the current stream) in one step; whatever they do not
        # take goes through the checks below
        bf16, i32 = torch.bfloat16, torch.int32
        store = ("storage", tuple((s, torch.uint8 if i % 2 == 0 else bf16) for i, s in enumerate(self.storage_shapes())))
        meta = (("in", self._table_shape, None, i32), ("in", (batch,), None, i32), ("maybe", (batch,), None, i32))
        kv, kv_out = ("in", self._kv_shape, None, bf16), ("out", self._kv_shape, bf16)
        self._write = _planned_call("kv_cache_write", h, (kv, kv, store, *meta))
        self._read = _planned_call("kv_cache_read", h, (store, *meta, kv_out, kv_out))
        self._attend = None
        if self._workspace_bytes is not None:
            self._attend = _planned_call("kv_cache_attend", h, (("in", self._q_shape, None, bf16), store, *meta,
                                                                ("out", self._o_shape, bf16),
                                                                ("workspace", self._workspace_bytes)))
        self._call = _planned_call_function()

    def storage_shapes(self):
        """Shapes of (k_codes, k_params, v_codes, v_params): codes uint8, params bfloat16 (scale, zero)."""
        return self._codes_shape, self._params_shape, self._codes_shape, self._params_shape

    def alloc_storage(self, device):
        """The cache's memory, every row standing for zeros."""
        return tuple(torch.zeros(s, dtype=torch.uint8 if i % 2 == 0 else torch.bfloat16, device=device)
                     for i, s in enumerate(self.storage_shapes()))

    def workspace_bytes(self) -> int:
        """Device workspace ``attend`` needs."""
        if self._workspace_bytes is None:
            raise FusedProjError(self._lib.kv_cache_attend_workspace_size(self._h, ctypes.byref(ctypes.c_size_t())),
                                 "kv_cache_attend_workspace_size")
        return self._workspace_bytes

    def alloc_workspace(self, device) -> torch.Tensor:
        return torch.empty((self.workspace_bytes(),), dtype=torch.uint8, device=device)

    def _check(self, name, t, shape, dtype, device):
        if t is None or t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on {device}")

    def _cache(self, storage, table, lengths, counts, device):
        if device.type != "cuda":
            raise TypeError("the cache and its inputs are GPU tensors")
        if device.index != self._device:
            raise ValueError(f"the plan is for cuda:{self._device}, not for {device}")
        kc, kp, vc, vp = storage
        self._check("k_codes", kc, self._codes_shape, torch.uint8, device)
        self._check("k_params", kp, self._params_shape, torch.bfloat16, device)
        self._check("v_codes", vc, self._codes_shape, torch.uint8, device)
        self._check("v_params", vp, self._params_shape, torch.bfloat16, device)
        self._check("table", table, self._table_shape, torch.int32, device)
        self._check("lengths", lengths, (self.B,), torch.int32, device)
        if counts is not None:
            self._check("counts", counts, (self.B,), torch.int32, device)
        return ctypes.byref(KVCacheStorage(kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr()))

    def write(self, storage, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
              counts: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> None:
        if stream is None and self._write is not None:
            r = self._call(self._write, k, v, storage, table, lengths, counts, None)
            if type(r) is tuple:
                return
            if r is not None:
                raise FusedProjError(r, "kv_cache_write")
        dev = k.device
        s = self._cache(storage, table, lengths, counts, dev)
        self._check("k", k, self._kv_shape, torch.bfloat16, dev)
        self._check("v", v, self._kv_shape, torch.bfloat16, dev)
        st = stream if stream is not None else torch.cuda.current_stream(dev)
        rc = self._lib.kv_cache_write(self._h, k.data_ptr(), v.data_ptr(), s, table.data_ptr(), lengths.data_ptr(),
                                      None if counts is None else counts.data_ptr(), st.cuda_stream)
        if rc != OK:
            raise FusedProjError(rc, "kv_cache_write")

    def read(self, storage, table: torch.Tensor, lengths: torch.Tensor, counts: torch.Tensor | None = None, out=None,
             stream: torch.cuda.Stream | None = None):
        """(k, v) [batch*KVH, tokens, hd] of the step's tokens, zeros for padding and absent pages. With
        counts = lengths that is all the cache holds, from position 0."""
        if out is None and stream is None and self._read is not None:
            r = self._call(self._read, storage, table, lengths, counts, None)
            if type(r) is tuple:
                return r
            if r is not None:
                raise FusedProjError(r, "kv_cache_read")
        dev = table.device
        s = self._cache(storage, table, lengths, counts, dev)
        if out is None:
            with _allocate_on(stream):
                k = torch.empty(self._kv_shape, dtype=torch.bfloat16, device=dev)
                v = torch.empty(self._kv_shape, dtype=torch.bfloat16, device=dev)
        else:
            k, v = out
            self._check("k", k, self._kv_shape, torch.bfloat16, dev)
            self._check("v", v, self._kv_shape, torch.bfloat16, dev)
        st = stream if stream is not None else torch.cuda.current_stream(dev)
        rc = self._lib.kv_cache_read(self._h, s, table.data_ptr(), lengths.data_ptr(),
                                     None if counts is None else counts.data_ptr(), k.data_ptr(), v.data_ptr(),
                                     st.cuda_stream)
        if rc != OK:
            raise FusedProjError(rc, "kv_cache_read")
        return k, v

    def attend(self, storage, q: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
               counts: torch.Tensor | None = None, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
        """Attention of the step's queries; the workspace (uint8 device tensor of at least
        workspace_bytes()) is allocated when not given."""
        if out is None and stream is None and self._attend is not None:
            r = self._call(self._attend, q, storage, table, lengths, counts, workspace)
            if type(r) is tuple:
                return r[0]
            if r is not None:
                raise FusedProjError(r, "kv_cache_attend")
        need = self.workspace_bytes()
        dev = q.device
        s = self._cache(storage, table, lengths, counts, dev)
        self._check("q", q, self._q_shape, torch.bfloat16, dev)
        if out is None or workspace is None and need:
            with _allocate_on(stream):
                if out is None:
                    out = torch.empty(self._o_shape, dtype=torch.bfloat16, device=dev)
                if workspace is None:
                    workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
        self._check("out", out, self._o_shape, torch.bfloat16, dev)
        if need and (workspace.device != dev or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        st = stream if stream is not None else torch.cuda.current_stream(dev)
        rc = self._lib.kv_cache_attend(self._h, q.data_ptr(), s, table.data_ptr(), lengths.data_ptr(),
                                       None if counts is None else counts.data_ptr(), out.data_ptr(),
                                       workspace.data_ptr() if need else None,
                                       workspace.numel() * workspace.element_size() if need else 0, st.cuda_stream)
        if rc != OK:
            raise FusedProjError(rc, "kv_cache_attend")
        return out

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._write = self._read = self._attend = None
            self._lib.kv_cache_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
