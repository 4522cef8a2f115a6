"""Attention over whole prompts: descriptor, refusals, exports, and its reference's gradients, without a GPU."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import attention_reference as ref
import ff_input_projection_amd as fpa
from ff_input_projection_amd import PromptAttention, make_prompt_attention_desc, validate_prompt_attention

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_exports_what_the_header_declares():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "prompt_attention.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b(prompt_attention_[a-z_]+)\s*\(", text))
    assert declared == set(fpa.PROMPT_ATTENTION_SYMBOLS)
    lib = fpa.load_library()
    for name in declared:
        assert hasattr(lib, name), name


def test_descriptor_layout_matches_c(tmp_path):
    src = ('#include <stdio.h>\n#include <stddef.h>\n#include "prompt_attention.h"\n'
           'int main(void){printf("%zu %zu %zu %zu %zu\\n", sizeof(prompt_attention_desc), offsetof(prompt_attention_desc, batch), '
           'offsetof(prompt_attention_desc, q_strides), offsetof(prompt_attention_desc, v_strides), '
           'offsetof(prompt_attention_desc, sm_scale)); return 0;}\n')
    exe = str(tmp_path / "layout")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-x", "c", "-",
                        "-o", exe], input=src, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    vals = list(map(int, subprocess.run([exe], capture_output=True, text=True).stdout.split()))
    D = fpa.PromptAttentionDesc
    assert vals == [ctypes.sizeof(D), D.batch.offset, D.q_strides.offset, D.v_strides.offset, D.sm_scale.offset]


def _desc(batch=2, tokens=5, n_heads=8, head_dim=64, **kw):
    return make_prompt_attention_desc(batch, tokens, n_heads, head_dim, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(), fpa.OK), (dict(batch=0), fpa.OK), (dict(n_kv_heads=2), fpa.OK), (dict(causal=False), fpa.OK),
    (dict(head_dim=8), fpa.OK), (dict(head_dim=256), fpa.OK), (dict(batch=1, sequences=7), fpa.OK),
    (dict(q_strides=(0, 64, 0)), fpa.OK), (dict(k_strides=(8, 8, 1 << 24)), fpa.OK), (dict(sm_scale=1e-30), fpa.OK),
    (dict(tokens=0), fpa.EINVAL), (dict(batch=-1), fpa.EINVAL), (dict(n_heads=0), fpa.EINVAL), (dict(head_dim=0), fpa.EINVAL),
    (dict(n_kv_heads=3), fpa.EINVAL), (dict(n_kv_heads=-1), fpa.EINVAL), (dict(sequences=2), fpa.EINVAL),
    (dict(batch=1, sequences=-1), fpa.EINVAL), (dict(v_strides=(320, -64, 64)), fpa.EINVAL),
    (dict(sm_scale=-1.0), fpa.EINVAL), (dict(sm_scale=float("inf")), fpa.EINVAL), (dict(sm_scale=float("nan")), fpa.EINVAL),
    (dict(sm_scale=2.3e38), fpa.OK), (dict(sm_scale=2.4e38), fpa.EINVAL), (dict(sm_scale=1e-39), fpa.EINVAL),
    (dict(dtype=torch.float32), fpa.EUNSUPPORTED), (dict(head_dim=20), fpa.EUNSUPPORTED), (dict(head_dim=264), fpa.EUNSUPPORTED),
    (dict(q_strides=(320, 64, 68)), fpa.EUNSUPPORTED), (dict(k_strides=(8, 8, (1 << 24) + 8)), fpa.EUNSUPPORTED),
    (dict(k_strides=(1 << 60, 8, 8)), fpa.EUNSUPPORTED), (dict(tokens=1 << 30), fpa.EUNSUPPORTED),
    (dict(batch=1, sequences=1 << 30), fpa.EUNSUPPORTED), (dict(batch=1 << 20, tokens=1 << 12), fpa.EUNSUPPORTED),
    (dict(n_heads=1 << 40), fpa.EUNSUPPORTED), (dict(n_heads=1 << 19), fpa.EUNSUPPORTED), (dict(n_heads=1 << 18), fpa.OK),
    # launches of 2^32 threads
    (dict(batch=1 << 20, tokens=1), fpa.EUNSUPPORTED), (dict(batch=(1 << 20) - 1, tokens=1), fpa.OK),
    (dict(batch=1 << 18, tokens=200), fpa.EUNSUPPORTED), (dict(batch=(1 << 18) - 1, tokens=200), fpa.OK),
])
def test_validate(kw, code):
    assert validate_prompt_attention(_desc(**kw)) == code


def test_wrong_enums_and_null():
    lib = fpa.load_library()
    assert lib.prompt_attention_validate(None) == fpa.EINVAL
    for field, value in (("dtype", 7), ("causal", 2), ("causal", -1)):
        d = _desc()
        setattr(d, field, value)
        assert validate_prompt_attention(d) == fpa.EINVAL, field
    assert lib.prompt_attention_create(ctypes.byref(_desc()), None) == fpa.EINVAL
    assert lib.prompt_attention_destroy(None) == fpa.OK
    n = ctypes.c_size_t()
    assert lib.prompt_attention_backward_workspace_size(None, ctypes.byref(n)) == fpa.EINVAL
    assert lib.prompt_attention_run(*[None] * 8) == fpa.EINVAL
    assert lib.prompt_attention_backward(*[None] * 12, 0, None) == fpa.EINVAL


def test_python_refusals():
    with pytest.raises(KeyError):
        _desc(dtype=torch.float16)
    with pytest.raises(fpa.FusedProjError):
        PromptAttention(2, 5, 8, 20)
    x = torch.empty((6, 5, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        PromptAttention.for_tensors(x, x, x, batch=4)
    with pytest.raises(ValueError):
        PromptAttention.for_tensors(x, x[None], x)
    with pytest.raises(ValueError):
        PromptAttention.for_tensors(x[None], x[None], x[None].transpose(2, 3))


@pytest.mark.parametrize("causal", [True, False])
def test_the_reference_is_the_gradient(causal):
    """Central differences of sum(do o) in 64 bits: off by h^2 and by the sums' roundings over h."""
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((1, 4, 9, 8)), rng.standard_normal((1, 2, 9, 8)), rng.standard_normal((1, 2, 9, 8))
    do = rng.standard_normal((1, 9, 4, 8))
    where = ref.spans(1, 9, 3, [1, 4, 4, 8])
    got = ref.attention(q, k, v, causal, 0.3, where, do)
    loss = lambda: (ref.attention(q, k, v, causal, 0.3, where)["o"][0] * do).sum()
    h = 1e-4
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for at in rng.integers(0, x.size, 40):
            old = x.flat[at]
            x.flat[at] = old + h
            above = loss()
            x.flat[at] = old - h
            below = loss()
            x.flat[at] = old
            assert abs((above - below) / (2 * h) - got[name][0].flat[at]) < 1e-6
