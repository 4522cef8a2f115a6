"""The quantised key/value cache and the attention over it on the GPU: stored bytes and values read back bit for bit
against the definition, attention against the definition in 64 bits (the bound is derived in kv_reference.attend)."""
import math

import numpy as np
import pytest
import torch

import kv_reference as ref
from ff_input_projection_amd import (EALIAS, EALIGN, EINVAL, FusedProjection, FusedProjError, KVCache, LayerNorm,
                                     SplitRope)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = dict(dtype=torch.int32, device=DEV)


class Case:
    """A cache with random pages and what is in it, on both sides."""

    def __init__(self, bits, batch, tokens, heads, kvh, hd, page, max_pages, lengths, counts, seed=0, table=None, scale=0.0):
        self.bits, self.batch, self.tokens, self.heads, self.kvh, self.hd = bits, batch, tokens, heads, kvh, hd
        self.page, self.lengths, self.counts = page, lengths, counts
        self.g = torch.Generator().manual_seed(seed)
        self.n_pages = batch * max_pages + 2
        self.capacity = max_pages * page
        self.table = torch.randperm(self.n_pages, generator=self.g)[:batch * max_pages].view(batch, max_pages).to(torch.int32)
        if table is not None:
            table(self.table)
        kw = dict(n_kv_heads=kvh, bits=bits, page_size=page, n_pages=self.n_pages, max_pages=max_pages, sm_scale=scale)
        self.plan = KVCache(batch, tokens, heads, hd, **kw)
        self.whole = KVCache(batch, self.capacity, kvh, hd, **kw)     # writes and reads any length at once
        self.scale = scale or hd ** -0.5
        self.args = (self.table.to(DEV), torch.tensor(lengths, **I32), None if counts is None else torch.tensor(counts, **I32))

    def random(self, *shape):
        """bf16 rows whose channels differ in width and offset."""
        x = torch.randn(shape, generator=self.g, dtype=torch.float64)
        off = torch.randn(shape[-1], generator=self.g, dtype=torch.float64) * (torch.arange(shape[-1]) % 7 == 3) * 3
        return (x + off).to(torch.bfloat16)

    def dirty_storage(self):
        """Memory whose every slot holds the largest codes and NaN: nothing of it may show."""
        st = self.plan.alloc_storage(DEV)
        for t in st:
            t.fill_(255 if t.dtype == torch.uint8 else float("nan"))
        return st

    def fill(self, storage, k=None, v=None):
        """Writes whole sequences ([batch, kvh, capacity, hd]) and keeps their (code, scale, zero)."""
        shape = (self.batch, self.kvh, self.capacity, self.hd)
        k = self.random(*shape) if k is None else k
        v = self.random(*shape) if v is None else v
        n = torch.tensor([min(max(x, 0), self.capacity) for x in self.lengths], **I32)
        self.whole.write(storage, k.view(-1, *shape[2:]).to(DEV), v.view(-1, *shape[2:]).to(DEV), self.args[0], n, n)
        self.rows = [ref.quantise(x, self.bits) for x in (k, v)]

    def expected(self, q):
        """(o, tolerance) [batch, tokens, H, hd]."""
        out = []
        gone = (self.table < 0) | (self.table >= self.n_pages)
        q64 = q.double().numpy().reshape(self.batch, self.heads, self.tokens, self.hd)
        for i in range(self.batch):
            length = min(max(self.lengths[i], 0), self.capacity)
            own = ref.positions(self.lengths[i], None if self.counts is None else self.counts[i], self.tokens, 1 << 40)
            own = {s: p for s, p in own.items()}
            k, v = ([c[i].astype(np.float64), s[i].astype(np.float64), z[i].astype(np.float64)] for c, s, z in self.rows)
            k[1] = np.where(gone[i].numpy().repeat(self.page)[None, :], -1.0, k[1])
            out.append(ref.attend(q64[i], k, v, own, length, self.heads // self.kvh, self.scale,
                                  self.bits))
        return np.stack([o for o, _ in out]), np.stack([t for _, t in out])

    def queries(self):
        return self.random(self.batch * self.heads, self.tokens, self.hd)

    def attend(self, storage, q, **kw):
        """Into an output and with a workspace full of NaN."""
        out = torch.full((self.batch, self.tokens, self.heads * self.hd), float("nan"), dtype=torch.bfloat16, device=DEV)
        ws = torch.full((self.plan.workspace_bytes() // 4,), float("nan"), device=DEV)
        self.plan.attend(storage, q.to(DEV), *self.args, out=out, workspace=ws, **kw)
        torch.cuda.synchronize()
        return out.double().cpu().numpy().reshape(self.batch, self.tokens, self.heads, self.hd)


def within(got, want, tol):
    assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN in other places"
    fine = ~np.isnan(want)
    err = np.abs(got[fine] - want[fine])
    print(f"[kv_cache] max err/tol {(err / np.maximum(tol[fine], 1e-300)).max(initial=0.0):.3g}", flush=True)
    assert (err <= tol[fine]).all()


# ------------------------------------------------------------------------------------------------ write and read
ROWS = [  # bits, batch, tokens, kvh, hd, page, max_pages, lengths, counts
    (4, 1, 1, 1, 8, 16, 1, [1], None), (8, 1, 1, 1, 8, 16, 1, [16], None),
    (4, 3, 1, 2, 128, 64, 3, [1, 64, 65], None), (8, 3, 1, 2, 128, 64, 3, [192, 128, 1], [1, 0, 1]),
    (4, 4, 37, 5, 64, 16, 4, [37, 64, 20, 0], [37, 5, 20, 0]), (8, 4, 37, 5, 64, 16, 4, [40, 64, 20, 1], [37, 30, 0, 1]),
    (4, 2, 50, 3, 96, 48, 3, [144, 51], [50, 49]), (8, 2, 50, 3, 96, 48, 3, [144, 51], [50, 49]),
    (4, 2, 9, 1, 256, 32, 2, [9, 33], None), (8, 2, 9, 1, 512, 32, 2, [64, 33], None), (4, 2, 7, 2, 24, 16, 2, [9, 32], [7, 7]),
    (8, 1, 130, 2, 32, 16, 40, [600], None), (4, 1, 130, 2, 40, 16, 40, [600], None),
    # what lengths and counts should not hold: below 0, past the capacity, more than the step
    (4, 4, 6, 2, 32, 16, 2, [-5, 40, 30, 3], [3, 6, -2, 99]), (8, 3, 6, 2, 32, 16, 2, [2, 35, 2 ** 31 - 1], [6, 6, 6]),
]


def _rows_case(bits, batch, tokens, kvh, hd, page, max_pages, lengths, counts, seed=0, table=None):
    return Case(bits, batch, tokens, kvh, kvh, hd, page, max_pages, lengths, counts, seed, table)


def _check_rows(c, k, v):
    """Writes, compares every byte of the storage, reads back, compares every bit."""
    storage = c.plan.alloc_storage(DEV)
    for t in storage:
        t.view(torch.uint8).fill_(0xA5)
    want = [t.cpu() for t in storage]
    back = [torch.zeros((c.batch, c.kvh, c.tokens, c.hd), dtype=torch.bfloat16) for _ in range(2)]
    for n, x in enumerate((k, v)):
        code, scale, zero = ref.quantise(x, c.bits)
        packed = torch.from_numpy(ref.pack(code, c.bits))
        params = torch.from_numpy(np.stack([scale, zero], -1)).to(torch.bfloat16)
        with np.errstate(all="ignore"):
            value = zero[..., None] + scale[..., None] * code.astype(np.float32)
        value = torch.from_numpy(value).to(torch.bfloat16)
        for i in range(c.batch):
            for s, p in ref.positions(c.lengths[i], None if c.counts is None else c.counts[i], c.tokens, c.capacity).items():
                page = int(c.table[i, p // c.page])
                if 0 <= page < c.n_pages:
                    want[2 * n][page, :, p % c.page] = packed[i, :, s]
                    want[2 * n + 1][page, :, p % c.page] = params[i, :, s]
                    back[n][i, :, s] = value[i, :, s]
    flat = (c.batch * c.kvh, c.tokens, c.hd)
    c.plan.write(storage, k.view(flat).to(DEV), v.view(flat).to(DEV), *c.args)
    out = tuple(torch.full(flat, 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c.plan.read(storage, *c.args, out=out)
    torch.cuda.synchronize()
    for got, w in zip(storage, want):
        got = got.cpu()
        if got.dtype == torch.bfloat16:
            assert torch.equal(torch.isnan(got), torch.isnan(w))
            got, w = got.nan_to_num(), w.nan_to_num()
            got, w = got.view(torch.int16), w.view(torch.int16)
        assert torch.equal(got, w)
    for got, w in zip(out, back):
        assert torch.equal(got.cpu().view(w.shape).nan_to_num(9.0), w.nan_to_num(9.0))
    return storage, out


@pytest.mark.parametrize("case", ROWS, ids=[f"{c[0]}bit_b{c[1]}_t{c[2]}_h{c[3]}x{c[4]}_p{c[5]}" for c in ROWS])
def test_write_and_read(case):
    print(f"[case] kv_cache rows {case}", flush=True)
    c = _rows_case(*case)
    shape = (c.batch, c.kvh, c.tokens, c.hd)
    _check_rows(c, c.random(*shape), c.random(*shape))


@pytest.mark.parametrize("bits", [4, 8])
def test_rows_at_the_borders(bits):
    """Constant rows, rows of two values, ties, the widest and the narrowest scales, rows with NaN or infinities."""
    c = _rows_case(bits, 1, 24, 1, 32, 16, 2, [24], None)
    k, v = c.random(1, 1, 24, 32), c.random(1, 1, 24, 32)
    k[0, 0, 0] = 3.0
    k[0, 0, 1] = 0.0
    k[0, 0, 2] = torch.where(torch.arange(32) % 2 == 0, -1.0, 2.0)
    k[0, 0, 3] = torch.arange(32) * 0.5                       # quotients that end in .5
    k[0, 0, 4] = torch.arange(32) * 2.0 ** -133               # denormal values
    k[0, 0, 5] = torch.arange(32) * 2.0 ** 18
    k[0, 0, 6] = torch.arange(32) * 2.0 ** 119                # a scale above 2^24
    k[0, 0, 7] = torch.where(torch.arange(32) == 9, 3.3e38, -3.3e38)
    k[0, 0, 8, 31] = float("nan")
    k[0, 0, 9, 0] = float("inf")
    k[0, 0, 10, 8] = float("-inf")
    k[0, 0, 11] = float("inf")
    k[0, 0, 12] = torch.arange(32) % 2 * (2.0 ** 24 * (2 ** bits - 1))   # the largest scale that is kept
    k[0, 0, 13] = torch.arange(32) % 2 * (2.0 ** 24 * (2 ** bits - 1)) * 1.02
    k[0, 0, 14] = 1000.0 + torch.arange(32) % 3 * 8.0
    k[0, 0, 15, 5] = -250.0
    v[0, 0, 3] = -0.0
    v[0, 0, 20, 4] = float("nan")
    _, (kb, vb) = _check_rows(c, k.to(torch.bfloat16), v)
    assert torch.isnan(kb[0, [6, 7, 8, 9, 10, 11, 13]]).all() and torch.isfinite(kb[0, [0, 1, 2, 3, 4, 5, 12, 14, 15]]).all()
    assert torch.equal(kb[0, :2].cpu(), k[0, 0, :2].to(torch.bfloat16))


@pytest.mark.parametrize("bits", [4, 8])
def test_pages_that_are_none(bits):
    def table(t):
        t[0, 1] = -1
        t[1, 0] = 2 ** 31 - 1
        t[1, 2] = 4 * 2 + 99
        t[2, :] = -2 ** 31

    c = _rows_case(bits, 3, 60, 2, 64, 16, 4, [64, 60, 61], [60, 60, 60], table=table)
    _check_rows(c, c.random(3, 2, 60, 64), c.random(3, 2, 60, 64))


# ------------------------------------------------------------------------------------------------ attention
ATTEND = [  # bits, batch, tokens, heads, kvh, hd, page, max_pages, lengths, counts
    (4, 1, 1, 1, 1, 32, 16, 1, [1], None), (8, 1, 1, 1, 1, 32, 16, 1, [1], None),
    (4, 2, 1, 8, 2, 128, 64, 3, [129, 192], None), (8, 2, 1, 8, 2, 128, 64, 3, [129, 192], None),
    (4, 5, 1, 4, 4, 64, 16, 30, [0, 1, 15, 33, 480], None), (8, 5, 1, 4, 4, 64, 16, 30, [0, 1, 15, 33, 480], None),
    (4, 3, 1, 32, 2, 64, 32, 20, [640, 31, 500], [1, 0, 1]),              # 16 heads of a group
    (4, 2, 1, 24, 1, 96, 48, 9, [432, 100], None), (8, 2, 1, 24, 1, 96, 48, 9, [432, 100], None),
    (4, 2, 1, 6, 2, 192, 16, 9, [144, 77], None), (8, 2, 1, 6, 2, 192, 16, 9, [144, 77], None),
    (4, 2, 1, 6, 1, 256, 16, 9, [144, 77], None), (8, 2, 1, 6, 1, 256, 16, 9, [144, 77], None),
    (4, 3, 5, 6, 2, 64, 16, 12, [190, 5, 3], [5, 5, 3]), (8, 3, 5, 6, 2, 64, 16, 12, [190, 5, 3], [5, 5, 3]),
    (4, 2, 7, 8, 2, 128, 64, 5, [300, 6], None),                          # 28 rows; a token before position 0
    (4, 2, 37, 4, 2, 32, 32, 7, [224, 37], [37, 20]), (8, 2, 37, 4, 2, 32, 32, 7, [224, 37], [37, 20]),
    (4, 1, 200, 8, 2, 128, 64, 8, [500], [190]), (8, 1, 200, 8, 2, 128, 64, 8, [500], [190]),
    (4, 1, 100, 3, 3, 96, 16, 8, [100], None), (4, 1, 65, 2, 1, 256, 16, 9, [140], None), (8, 1, 65, 2, 1, 192, 16, 9, [140], None),
    (4, 40, 70, 14, 7, 32, 16, 6, [96 - i for i in range(40)], [70 - i % 9 for i in range(40)]),       # rows over all waves
    (8, 40, 70, 14, 7, 64, 16, 6, [96 - 2 * i for i in range(40)], [min(70, 96 - 2 * i) for i in range(40)]),
    (4, 33, 33, 16, 8, 128, 16, 4, [64 - i for i in range(33)], [33 - i % 5 for i in range(33)]),
    (4, 50, 40, 6, 6, 192, 16, 3, [48 - i % 8 for i in range(50)], None),
    (8, 50, 40, 6, 6, 256, 16, 3, [48 - i % 8 for i in range(50)], None),
    (4, 3, 1, 8, 2, 128, 64, 40, [2560, 1, 1999], None), (8, 3, 1, 8, 2, 128, 64, 40, [2560, 1, 1999], None),   # joined parts
    (4, 2, 9, 6, 2, 96, 48, 50, [2400, 700], [9, 4]), (8, 1, 3, 2, 1, 256, 16, 100, [1600], None),
    (4, 1, 2, 8, 8, 32, 16, 200, [3200], None), (4, 1, 90, 4, 2, 64, 64, 30, [1900], None),
    (4, 2, 3, 4, 2, 64, 16, 3, [60, -4], [3, 3]), (4, 2, 3, 4, 2, 64, 16, 3, [48, 10], [77, -1]),   # what they should not hold
]


@pytest.mark.parametrize("case", ATTEND, ids=[f"{c[0]}bit_b{c[1]}_t{c[2]}_h{c[3]}of{c[4]}x{c[5]}_p{c[6]}" for c in ATTEND])
def test_attend(case):
    print(f"[case] kv_cache attend {case}", flush=True)
    c = Case(*case, seed=3)
    storage = c.dirty_storage()
    c.fill(storage)
    q = c.queries()
    within(c.attend(storage, q), *c.expected(q))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tokens", [1, 40])
def test_attend_over_absent_pages(bits, tokens):
    def table(t):
        t[0, 0] = -1
        t[0, 5] = 10 ** 6
        t[1, :] = -7

    c = Case(bits, 2, tokens, 6, 2, 64, 16, 8, [125, 128], None, seed=4, table=table)
    storage = c.dirty_storage()
    c.fill(storage)
    q = c.queries()
    o = c.attend(storage, q)
    within(o, *c.expected(q))
    assert not o[1].any()


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_attend_non_finite_values_reach_whoever_sees_them(tokens):
    c = Case(4, 3, tokens, 4, 2, 64, 16, 8, [120, 121, 122], None, seed=5)
    shape = (3, 2, 128, 64)
    k, v = c.random(*shape), c.random(*shape)
    k[0, 0, 118, 3] = float("nan")        # seen by the last two tokens of one k/v head
    v[1, 1, 60, 0] = float("inf")         # seen by every token of the other
    storage = c.dirty_storage()
    c.fill(storage, k, v)
    q = c.queries()
    qv = q.view(3, 4, tokens, 64)
    qv[2, 1, 0, 5], qv[2, 3, tokens - 1, 0] = float("nan"), float("-inf")
    want, tol = c.expected(q)
    want[2, tokens - 1, 3] = float("nan")
    o = c.attend(storage, q)
    within(o, want, tol)
    assert np.isnan(o[0, tokens - 1, :2]).all() and np.isfinite(o[0, :, 2:]).all()
    assert np.isnan(o[1, :, 2:]).all() and np.isfinite(o[1, :, :2]).all()
    assert np.isnan(o[2, 0, 1]).all() and np.isfinite(o[2, :, [0, 2]]).all()


@pytest.mark.parametrize("power", [-120, -60, 0, 20, 60, 89])
def test_attend_queries_of_any_size(power):
    """Scaled queries with the reverse in sm_scale: the same logits, whatever the power of two."""
    c = Case(4, 2, 3, 4, 2, 64, 16, 6, [90, 33], None, seed=6, scale=math.ldexp(0.125, -power))
    storage = c.dirty_storage()
    c.fill(storage)
    q = c.queries()
    q = (q * (1.9 / q.abs().max())).to(torch.bfloat16)
    big = torch.ldexp(q.float(), torch.tensor(power)).to(torch.bfloat16)
    within(c.attend(storage, big), *c.expected(big))


def test_attend_query_too_large_is_nan():
    c = Case(8, 1, 2, 2, 1, 32, 16, 2, [20], None, seed=7)
    storage = c.dirty_storage()
    c.fill(storage)
    q = c.queries()
    q.view(2, 2, 32)[1, 0, 4] = 2.0 ** 90
    want, tol = c.expected(q)
    want[0, 0, 1] = float("nan")
    within(c.attend(storage, q), want, tol)


@pytest.mark.parametrize("power", [-60, -20, 8, 20])
def test_attend_values_of_any_size(power):
    c = Case(4, 2, 1, 4, 2, 64, 16, 30, [470, 33], None, seed=8)
    storage = c.dirty_storage()
    shape = (2, 2, 480, 64)
    v = torch.ldexp(c.random(*shape).float(), torch.tensor(power)).to(torch.bfloat16)
    c.fill(storage, None, v)
    q = c.queries()
    within(c.attend(storage, q), *c.expected(q))


def test_attend_steep_logits():
    """Logits of hundreds, the greatest at the far end: the running maximum has to move, and once more."""
    c = Case(8, 2, 1, 4, 2, 64, 16, 40, [640, 555], None, seed=9, scale=4.0)
    shape = (2, 2, 640, 64)
    k = (c.random(*shape).float() * torch.linspace(0.1, 4.0, 640)[:, None]).to(torch.bfloat16)
    storage = c.dirty_storage()
    c.fill(storage, k)
    q = c.queries()
    within(c.attend(storage, q), *c.expected(q))


def test_offsets_past_32_bits():
    """A cache whose codes take more than 4 GiB, the sequence in its last pages."""
    n_pages, kvh, hd, page = 20000, 8, 256, 256
    plan = KVCache(1, 300, kvh, hd, bits=4, page_size=page, n_pages=n_pages, max_pages=2)
    storage = tuple(torch.empty(s, dtype=torch.uint8 if i % 2 == 0 else torch.bfloat16, device=DEV)
                    for i, s in enumerate(plan.storage_shapes()))
    assert storage[0].numel() > 2 ** 32
    small = Case(4, 1, 300, kvh, kvh, hd, page, 2, [300], None, seed=10)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], **I32)
    k, v = small.random(kvh, 300, hd).to(DEV), small.random(kvh, 300, hd).to(DEV)
    q = small.queries().to(DEV)
    near = small.plan.alloc_storage(DEV)
    plan.write(storage, k, v, table, small.args[1])
    small.plan.write(near, k, v, *small.args)
    for a, b in zip(plan.read(storage, table, small.args[1]), small.plan.read(near, *small.args)):
        assert torch.equal(a, b)
    assert torch.equal(plan.attend(storage, q, table, small.args[1]), small.plan.attend(near, q, *small.args))


# ------------------------------------------------------------------------------------------------ how it is used
def test_refusals():
    c = Case(4, 2, 3, 4, 2, 64, 16, 40, [500, 7], [3, 1])
    storage = c.plan.alloc_storage(DEV)
    c.fill(storage)
    k, v = (torch.zeros((4, 3, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q, o = torch.zeros((8, 3, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 3, 256), dtype=torch.bfloat16, device=DEV)
    lib, h, st = c.plan._lib, c.plan._h, torch.cuda.current_stream().cuda_stream
    import ctypes
    from ff_input_projection_amd import KVCacheStorage
    p = lambda t: t.data_ptr()
    store = KVCacheStorage(*(p(t) for t in storage))
    s = ctypes.byref(store)
    meta = tuple(p(t) for t in c.args)
    assert lib.kv_cache_write(h, None, p(v), s, *meta, st) == EINVAL
    assert lib.kv_cache_write(h, p(k), p(v), None, *meta, st) == EINVAL
    assert lib.kv_cache_write(h, p(k), p(v), s, None, *meta[1:], st) == EINVAL
    assert lib.kv_cache_write(h, p(k), p(v), s, meta[0], None, meta[2], st) == EINVAL
    assert lib.kv_cache_write(h, p(k) + 2, p(v), s, *meta, st) == EALIGN
    assert lib.kv_cache_write(h, p(k), p(v), s, meta[0] + 2, *meta[1:], st) == EALIGN
    assert lib.kv_cache_write(h, p(storage[0]), p(v), s, *meta, st) == EALIAS
    twice = KVCacheStorage(p(storage[0]), p(storage[1]), p(storage[0]), p(storage[3]))
    assert lib.kv_cache_write(h, p(k), p(v), ctypes.byref(twice), *meta, st) == EALIAS
    assert lib.kv_cache_read(h, s, *meta, p(k), p(k), st) == EALIAS
    assert lib.kv_cache_read(h, s, *meta, p(k), None, st) == EINVAL
    ws = c.plan.alloc_workspace(DEV)
    assert ws.numel() > 0
    assert lib.kv_cache_attend(h, p(q), s, *meta, p(q), p(ws), ws.numel(), st) == EALIAS
    assert lib.kv_cache_attend(h, p(q), s, *meta, p(ws), p(ws), ws.numel(), st) == EALIAS
    assert lib.kv_cache_attend(h, p(q), s, *meta, p(o), p(ws), ws.numel() - 16, st) == EINVAL
    assert lib.kv_cache_attend(h, p(q), s, *meta, p(o), None, 0, st) == EINVAL
    assert lib.kv_cache_attend(h, None, s, *meta, p(o), p(ws), ws.numel(), st) == EINVAL
    assert lib.kv_cache_attend(h, p(q), s, *meta, p(o) + 2, p(ws), ws.numel(), st) == EALIGN
    with pytest.raises(ValueError):
        c.plan.write(storage, k[:2], v, *c.args)
    with pytest.raises(ValueError):
        c.plan.write(storage, k, v, c.args[0].long(), *c.args[1:])
    with pytest.raises(ValueError):
        c.plan.write(storage, k, v, c.args[0].cpu(), *c.args[1:])
    with pytest.raises(ValueError):
        c.plan.attend(storage, q.float(), *c.args)
    with pytest.raises(ValueError):
        c.plan.attend(storage, q.transpose(0, 1).contiguous().transpose(0, 1), *c.args)
    with pytest.raises(ValueError):
        c.plan.attend(storage[:2] + storage[:1] + storage[1:2], q, *c.args, out=o[:1])
    with pytest.raises(FusedProjError):
        c.plan.attend(storage, q, *c.args, workspace=ws[:16])
    odd = KVCache(1, 1, 2, 40, n_pages=2, max_pages=1)      # a head size that the cache keeps and attention does not take
    with pytest.raises(FusedProjError):
        odd.workspace_bytes()
    with pytest.raises(FusedProjError):
        odd.attend(odd.alloc_storage(DEV), torch.zeros((2, 1, 40), dtype=torch.bfloat16, device=DEV),
                   torch.zeros((1, 1), **I32), torch.zeros((1,), **I32))
    torch.cuda.synchronize()


def test_no_sequences():
    plan = KVCache(0, 2, 4, 64, n_kv_heads=2, n_pages=3, max_pages=2)
    storage = plan.alloc_storage(DEV)
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)
    meta = (torch.empty((0, 2), **I32), torch.empty((0,), **I32))
    plan.write(storage, e(0, 2, 64), e(0, 2, 64), *meta)
    k, v = plan.read(storage, *meta)
    assert k.shape == v.shape == (0, 2, 64) and plan.attend(storage, e(0, 2, 64), *meta).shape == (0, 2, 256)


@pytest.mark.parametrize("max_pages", [30, 90])
@pytest.mark.parametrize("tokens", [1, 6])
def test_graph_replays_read_the_lengths_anew(tokens, max_pages):
    """A captured step (write and attend, one workspace) replayed with other inputs, lengths and pages: the eager bits."""
    c = Case(4, 3, tokens, 8, 2, 64, 16, max_pages, [400, 77, 200], None, seed=11)
    storage = c.plan.alloc_storage(DEV)
    c.fill(storage)
    table, lengths, _ = (t.clone() if t is not None else None for t in c.args)
    counts = torch.full((3,), tokens, **I32)
    kv = (6, tokens, 64)
    k, v = c.random(*kv).to(DEV), c.random(*kv).to(DEV)
    q = c.queries().to(DEV)
    out, ws = torch.empty((3, tokens, 512), dtype=torch.bfloat16, device=DEV), c.plan.alloc_workspace(DEV)
    assert ws.numel() > 0
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        c.plan.write(storage, k, v, table, lengths, counts)
        c.plan.attend(storage, q, table, lengths, counts, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for step in range(4):
        lengths.copy_(torch.tensor([401 + step, 78 + 50 * step, 0 if step == 2 else 201], **I32))
        counts.copy_(torch.tensor([tokens, min(tokens, 1 + step), 0 if step == 2 else 1], **I32))
        table[0, 28] = table[0, 29] = -1
        k.copy_(c.random(*kv))
        q.copy_(c.random(*q.shape))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        again = [t.clone() for t in storage]
        c.plan.write(again, k, v, table, lengths, counts)
        want = c.plan.attend(again, q, table, lengths, counts)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(storage, again))


@pytest.mark.parametrize("max_pages", [30, 90])
def test_two_streams_at_once(max_pages):
    c = Case(8, 4, 1, 8, 2, 128, 16, max_pages, [400, 480, 3, 222], None, seed=12)
    storage = c.plan.alloc_storage(DEV)
    c.fill(storage)
    q = c.queries().to(DEV)
    want = c.plan.attend(storage, q, *c.args)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(6):
        got += [c.plan.attend(storage, q, *c.args, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("bits", [4, 8])
def test_a_block_in_serving(bits):
    """Layer norm, projection with RoPE, cache, attention, output projection: a prompt of 20 and 13 tokens, then four single
    tokens, each attending over all that came before, against the same steps in 64 bits from the stored rows.

    The attention's bound holds for the q that the projection gave and the rows that the cache holds; the output projection's
    is the sum over its 256 products of |w| times the attention's bound, and its own bf16 rounding and fp32 sums."""
    b, dim, heads, kvh, hd, longest = 2, 128, 4, 2, 64, 24
    g = torch.Generator().manual_seed(13)
    rnd = lambda *s: torch.randn(s, generator=g)
    width = (heads + 2 * kvh) * hd
    w_in, w_out = (rnd(dim, width) / dim ** 0.5).to(torch.bfloat16).to(DEV), (rnd(heads * hd, dim) / 16).to(torch.bfloat16).to(DEV)
    gamma, beta = (1 + 0.1 * rnd(dim)).to(torch.bfloat16).to(DEV), (0.1 * rnd(dim)).to(torch.bfloat16).to(DEV)
    lengths_now, storage = [0, 0], None
    table = torch.tensor([[3, 0], [1, 4]], **I32)
    kw = dict(n_kv_heads=kvh, bits=bits, page_size=16, n_pages=5, max_pages=2)
    for tokens, counts in [(20, [20, 13])] + [(1, [1, 1])] * 4:
        x = rnd(b, tokens, dim).to(torch.bfloat16).to(DEV)
        norm = LayerNorm.for_tensor(x, "tokens_last")
        y, _ = norm(x, gamma, beta)
        plain = FusedProjection.for_tensor(y, "tokens_last", ff_dim=width)
        qkv = plain(y, w_in)[0]
        # the sequences are at different positions: one rotation a sequence
        parts = [SplitRope(1, tokens, heads, hd, n_kv_heads=kvh, pos_offset=lengths_now[i])(qkv[i:i + 1].contiguous()) for i in range(b)]
        q, k, v = (torch.cat([p[n] for p in parts]) for n in range(3))
        lengths_now = [a + n for a, n in zip(lengths_now, counts)]
        meta = (table, torch.tensor(lengths_now, **I32), torch.tensor(counts, **I32))
        cache = KVCache(b, tokens, heads, hd, **kw)
        storage = cache.alloc_storage(DEV) if storage is None else storage
        cache.write(storage, k, v, *meta)
        o = cache.attend(storage, q, *meta)
        out_plan = FusedProjection.for_tensor(o, "tokens_last", ff_dim=dim)
        out = out_plan(o, w_out)[0]
        torch.cuda.synchronize()

        rows = []
        for codes, params in (storage[:2], storage[2:]):
            c = codes.cpu().numpy()
            c = c if bits == 8 else np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], hd)
            p = params.double().cpu().numpy()
            at = table.cpu().numpy()
            order = lambda a: a[at].transpose(0, 2, 1, *range(3, a.ndim + 1)).reshape(b, kvh, 32, *a.shape[3:])
            rows.append((order(c).astype(np.float64), order(p[..., 0]), order(p[..., 1])))
        q64 = q.double().cpu().numpy().reshape(b, heads, tokens, hd)
        for i in range(b):
            own = ref.positions(lengths_now[i], counts[i], tokens, 32)
            want, tol = ref.attend(q64[i], *([a[i] for a in r] for r in rows), own, lengths_now[i], heads // kvh, hd ** -0.5, bits)
            within(o[i].double().cpu().numpy().reshape(tokens, heads, hd), want, tol)
            w = w_out.double().cpu().numpy()
            flat, ftol = want.reshape(tokens, -1), tol.reshape(tokens, -1)
            bound = ftol @ np.abs(w) + 2.0 ** -8 * np.abs(flat @ w) + (256 + 8) * ref.U * (np.abs(flat) @ np.abs(w)) * 2
            within(out[i].double().cpu().numpy(), flat @ w, bound + 2.0 ** -8 * (ftol @ np.abs(w)))


def test_tensors_of_another_device_are_refused(monkeypatch):
    """A plan made where another device was current takes no tensors of this one."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    plan = KVCache(1, 1, 2, 64, n_pages=2, max_pages=1)
    monkeypatch.undo()
    storage = plan.alloc_storage(DEV)
    k, v, q = (torch.zeros((2, 1, 64), dtype=torch.bfloat16, device=DEV) for _ in range(3))
    meta = (torch.zeros((1, 1), **I32), torch.ones((1,), **I32))
    with pytest.raises(ValueError):
        plan.write(storage, k, v, *meta)
    with pytest.raises(ValueError):
        plan.read(storage, *meta)
    with pytest.raises(ValueError):
        plan.attend(storage, q, *meta)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tokens", [3, 40])
@pytest.mark.parametrize("where", ["padding", "head"])
def test_attend_queries_of_different_sizes_side_by_side(where, tokens, bits):
    """Rows of up to 2^89 beside ordinary and small ones: in the padding's place they do not show at all, as another head's
    they leave the others' accuracy (whose bound knows nothing of them)."""
    c = Case(bits, 2, tokens, 4, 2, 64, 16, 8, [120, 121], [tokens - 1, tokens - 2], seed=11)
    storage = c.dirty_storage()
    c.fill(storage)
    q = c.queries()
    qv = q.view(2, 4, tokens, 64)
    qv[:, 3] *= 2.0 ** -6
    clean = c.attend(storage, q)
    if where == "padding":
        qv[0, :, tokens - 1:] = 1.5 * 2.0 ** 89
        qv[1, :, tokens - 2:] = 1.5 * 2.0 ** 89
        o = c.attend(storage, q)
        within(o, *c.expected(q))
        assert np.array_equal(o, clean)
    else:
        qv[:, 2] *= 2.0 ** 80
        o = c.attend(storage, q)
        want, tol = c.expected(q)
        rest = [0, 1, 3]
        within(o[:, :, rest], want[:, :, rest], tol[:, :, rest])
        assert np.isfinite(o).all()


def test_captured_calls_that_allocate():
    """A step captured without outputs or workspaces of its own, on another stream than the default one: each replay gives
    the eager step's bits, for new contents of the same tensors too."""
    b, H, KVH, hd, page, pages = 3, 8, 2, 64, 16, 30
    g = torch.Generator(device=DEV).manual_seed(12)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)
    plan = KVCache(b, 1, H, hd, n_kv_heads=KVH, page_size=page, n_pages=b * pages, max_pages=pages)
    assert plan.workspace_bytes() > 0
    storage = plan.alloc_storage(DEV)
    table = torch.randperm(b * pages, generator=g, device=DEV).view(b, pages).to(torch.int32)
    x, gamma, beta = rand(b, 1, H * hd), rand(H * hd), rand(H * hd)
    norm = LayerNorm.for_tensor(x, "tokens_last")
    lengths = torch.tensor([1, 400, 479], **I32)
    k, v = rand(b * KVH, 1, hd), rand(b * KVH, 1, hd)

    def step():
        y, stats = norm(x, gamma, beta)
        plan.write(storage, k, v, table, lengths)
        o = plan.attend(storage, y.view(b * H, 1, hd), table, lengths)
        return (y, stats, o, *plan.read(storage, table, lengths), *norm.backward(x, gamma, stats, o))

    for n in (400, 470):     # something to look back at
        plan.write(storage, rand(b * KVH, 1, hd), rand(b * KVH, 1, hd), table, torch.full((b,), n, **I32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = step()
    torch.cuda.current_stream().wait_stream(side)
    for i in range(3):
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip(outs, want):
            assert torch.equal(a, e)
        x.copy_(rand(b, 1, H * hd))
        k.copy_(rand(b * KVH, 1, hd))
        lengths.add_(1 if i == 0 else 0)
        torch.cuda.synchronize()


LARGE_V = [  # bits, batch, tokens, heads, kvh, hd, page, max_pages, lengths: both kernels, one part and joined ones
    (4, 2, 1, 8, 2, 64, 16, 40, [640, 33]), (8, 1, 3, 2, 1, 256, 16, 100, [1600]), (4, 2, 1, 4, 2, 96, 16, 2, [30, 9]),
    (4, 1, 40, 4, 2, 128, 64, 40, [2560]), (8, 2, 200, 4, 4, 32, 64, 64, [4096, 4000]), (4, 1, 70, 2, 1, 192, 16, 9, [140]),
]


@pytest.mark.parametrize("power", [-100, 30, 40, 60, 100, 127])
@pytest.mark.parametrize("case", LARGE_V, ids=[f"{c[0]}bit_t{c[2]}_x{c[5]}" for c in LARGE_V])
def test_attend_constant_values_of_any_size(case, power):
    """Rows of one value are kept exactly (scale 0), whatever its size: alone in the first k/v head of the first sequence,
    beside ordinary rows and with both signs elsewhere."""
    c = Case(*case, None, seed=14)
    shape = (c.batch, c.kvh, c.capacity, c.hd)
    v = c.random(*shape)
    size = torch.tensor(1.5 * 2.0 ** power).to(torch.bfloat16)
    v[:, :, 0::2] = size
    v[:, :, 0::6] = -size
    v[0, 0] = size
    storage = c.dirty_storage()
    c.fill(storage, None, v)
    q = c.queries()
    want, tol = c.expected(q)
    within(c.attend(storage, q), want, tol)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tokens", [3, 40])
def test_attend_padding_beside_keys_of_large_scales(tokens, bits):
    """What lies in the padding's place of q does not show: not at the largest sizes either, over keys of scales of 2^14 and more."""
    c = Case(bits, 2, tokens, 4, 2, 64, 16, 8, [120, 121], [tokens - 1, tokens - 2], seed=15)
    storage = c.dirty_storage()
    c.fill(storage, c.random(2, 2, 128, 64) * 2.0 ** 20)
    q = c.queries() * 2.0 ** -20
    clean = c.attend(storage, q)
    within(clean, *c.expected(q))
    qv = q.view(2, 4, tokens, 64)
    for junk in (1.5 * 2.0 ** 89, float("nan"), 3.3e38):
        qv[0, :, tokens - 1:] = junk
        qv[1, :, tokens - 2:] = junk
        assert np.array_equal(c.attend(storage, q), clean)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tokens", [3, 40])
@pytest.mark.parametrize("sm_power", [-3, 5, 20])
def test_attend_large_queries_over_keys_of_large_scales(sm_power, tokens, bits):
    """A head's queries next to the bound of what is taken (2^90, or 2^96 over the logits' factor), over keys of scales
    of 2^14 and more: the other heads of the workgroup keep their accuracy, and the large ones have finite outputs."""
    c = Case(bits, 2, tokens, 4, 2, 64, 16, 8, [120, 121], None, seed=16, scale=2.0 ** sm_power)
    storage = c.dirty_storage()
    c.fill(storage, c.random(2, 2, 128, 64) * 2.0 ** 20)
    q = c.queries() * 2.0 ** (-23 - sm_power)                     # logits of ordinary size
    qv = q.view(2, 4, tokens, 64)
    largest = 89 - max(0, sm_power - 6)                           # log2(sm_scale log2 e) = sm_power + 0.53
    power = largest - math.frexp(float(qv[:, 2].abs().max()))[1]
    qv[:, 2] = torch.ldexp(qv[:, 2].float(), torch.tensor(power)).to(torch.bfloat16)
    assert 2.0 ** (largest - 1) <= qv[:, 2].abs().max() < 2.0 ** largest
    o = c.attend(storage, q)
    want, tol = c.expected(q)
    rest = [0, 1, 3]
    within(o[:, :, rest], want[:, :, rest], tol[:, :, rest])
    assert np.isfinite(o).all()


def test_attend_query_too_large_for_its_factor_is_nan():
    """With sm_scale log2(e) = 2^20.5 a value of 2^(96 - 20) is too large, one of half of that is not."""
    c = Case(4, 1, 2, 4, 1, 32, 16, 2, [20], None, seed=17, scale=2.0 ** 20)
    storage = c.dirty_storage()
    c.fill(storage)
    q = c.queries() * 2.0 ** -23
    qv = q.view(4, 2, 32)
    qv[1, 0, 4], qv[2, 1, 5] = 2.0 ** 76, -1.9375 * 2.0 ** 75
    o = c.attend(storage, q)
    want, tol = c.expected(q)
    assert np.isnan(o[0, 0, 1]).all() and np.isfinite(o[0, 1]).all()
    within(o[0, :, [0, 3]], want[0, :, [0, 3]], tol[0, :, [0, 3]])
