"""A wrong number of outputs is refused before anything reaches the library, which would take a surplus one as the argument
behind it (a workspace, a stream)."""
import pytest
import torch

from ff_input_projection_amd import PromptAttention, Rope

BF16 = torch.bfloat16
B, T, H, KVH, HD = 2, 6, 4, 2, 64


class NoLibrary:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was reached")


def plans(device):
    """A plan of each class; without a GPU, objects with what __init__ leaves."""
    if device == "cuda":
        return Rope(B, T, H, HD, n_kv_heads=KVH), PromptAttention(B, T, H, HD, n_kv_heads=KVH)
    rope, attention = Rope.__new__(Rope), PromptAttention.__new__(PromptAttention)
    for p in (rope, attention):
        p._lib, p._h, p._device = NoLibrary(), None, 0
        p.B, p.T, p.H, p.KVH, p.hd = B, T, H, KVH, HD
    rope.dtype = BF16
    rope._rows_shape, rope._q_shape, rope._kv_shape = rope.shapes()
    attention.sequences, attention._workspace_bytes = 0, 1024
    attention._shapes, attention._strides = [rope._q_shape, rope._kv_shape, rope._kv_shape], [None] * 3
    attention._o_shape, attention._lse_shape, attention._extents_shape = (B, T, H * HD), (B * H, T), (B,)
    return rope, attention


def check(device):
    rope, attention = plans(device)
    new = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device="cuda:0")
    rows, q, k, v = new(B, T, (H + 2 * KVH) * HD), new(B * H, T, HD), new(B * KVH, T, HD), new(B * KVH, T, HD)
    o, lse, ws = new(B, T, H * HD), new(B * H, T, dtype=torch.float32), new(1 << 20, dtype=torch.uint8)
    a, b, c = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for out in ((a, b), (a, b, c, ws), (), [a, b, c, None]):
        with pytest.raises(ValueError):
            rope(rows, out=out)
        with pytest.raises(ValueError):
            attention.backward(q, k, v, o, lse, o.clone(), out=out, workspace=ws)
    for out in ((a,), (a, b, c), (q, k, v), ()):        # (q, k, v): what the split is given
        with pytest.raises(ValueError):
            rope.rotate(q, k, out=out)
        with pytest.raises(ValueError):
            rope.rotate_backward(q, k, out=out)
    for out in ((o,), (o.clone(), lse, a), ()):
        with pytest.raises(ValueError):
            attention(q, k, v, out=out)


def test_a_wrong_number_of_outputs():
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        check("none")


@pytest.mark.gpu
def test_a_wrong_number_of_outputs_on_the_gpu():
    check("cuda")
