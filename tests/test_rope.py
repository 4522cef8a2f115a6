"""Rotary positions' descriptor, refusals and exports, without a GPU."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import ff_input_projection_amd as fpa
from ff_input_projection_amd import Rope, make_rope_desc, validate_rope

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_exports_what_the_header_declares():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "rope.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b(rope_[a-z_]+)\s*\(", text))
    assert declared == set(fpa.ROPE_SYMBOLS)
    lib = fpa.load_library()
    for name in declared:
        assert hasattr(lib, name), name


def test_descriptor_layout_matches_c(tmp_path):
    src = ('#include <stdio.h>\n#include <stddef.h>\n#include "rope.h"\n'
           'int main(void){printf("%zu %zu %zu %zu %zu\\n", sizeof(rope_desc), offsetof(rope_desc, tokens), '
           'offsetof(rope_desc, scaling), offsetof(rope_desc, original_tokens), offsetof(rope_desc, magnitude)); return 0;}\n')
    exe = str(tmp_path / "layout")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-x", "c", "-",
                        "-o", exe], input=src, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    vals = list(map(int, subprocess.run([exe], capture_output=True, text=True).stdout.split()))
    D = fpa.RopeDesc
    assert vals == [ctypes.sizeof(D), D.tokens.offset, D.scaling.offset, D.original_tokens.offset, D.magnitude.offset]


def _desc(batch=2, tokens=5, n_heads=8, head_dim=64, **kw):
    return make_rope_desc(batch, tokens, n_heads, head_dim, **kw)


BY_PARTS = dict(scaling="by_parts", factor=4.0, original_tokens=2048)


@pytest.mark.parametrize("kw,code", [
    (dict(), fpa.OK), (dict(batch=0), fpa.OK), (dict(n_kv_heads=2), fpa.OK), (dict(dtype=torch.float32), fpa.OK),
    (dict(pairs="interleaved"), fpa.OK), (dict(rope_dims=2), fpa.OK), (dict(rope_dims=62), fpa.OK),
    (dict(head_dim=4096), fpa.OK), (dict(scaling="linear", factor=0.5), fpa.OK), (BY_PARTS, fpa.OK),
    (dict(factor=float("nan")), fpa.OK),                                           # not used
    (dict(magnitude=0.0), fpa.OK), (dict(magnitude=-1.5), fpa.OK),
    (dict(tokens=0), fpa.EINVAL), (dict(batch=-1), fpa.EINVAL), (dict(n_heads=0), fpa.EINVAL),
    (dict(n_kv_heads=3), fpa.EINVAL), (dict(n_kv_heads=-1), fpa.EINVAL), (dict(head_dim=0), fpa.EINVAL),
    (dict(rope_dims=7), fpa.EINVAL), (dict(rope_dims=66), fpa.EINVAL), (dict(rope_dims=-2), fpa.EINVAL),
    (dict(rope_base=0.0), fpa.EINVAL), (dict(rope_base=float("inf")), fpa.EINVAL), (dict(rope_base=float("nan")), fpa.EINVAL),
    (dict(magnitude=float("inf")), fpa.EINVAL), (dict(magnitude=1e39), fpa.EINVAL),
    (dict(scaling="linear", factor=0.0), fpa.EINVAL), (dict(scaling="linear", factor=float("inf")), fpa.EINVAL),
    ({**BY_PARTS, "original_tokens": 0}, fpa.EINVAL), ({**BY_PARTS, "low_turns": 32.0}, fpa.EINVAL),
    ({**BY_PARTS, "high_turns": float("nan")}, fpa.EINVAL),
    # angles that extended precision does not hold at far positions
    (dict(rope_base=0.5), fpa.OK), (dict(rope_base=0.1), fpa.EUNSUPPORTED), (dict(rope_base=1e-300), fpa.EUNSUPPORTED),
    (dict(scaling="by_parts", factor=1e-3, original_tokens=1), fpa.EUNSUPPORTED),
    (dict(scaling="linear", factor=0.125), fpa.OK), (dict(scaling="linear", factor=0.124), fpa.EUNSUPPORTED),
    (dict(head_dim=20), fpa.EUNSUPPORTED), (dict(head_dim=4104), fpa.EUNSUPPORTED),
    (dict(n_heads=1 << 15), fpa.EUNSUPPORTED), (dict(n_heads=1 << 62), fpa.EUNSUPPORTED),
    (dict(tokens=1 << 31), fpa.EUNSUPPORTED), (dict(batch=1, tokens=(1 << 25) - 1), fpa.OK),
    (dict(batch=1, tokens=1 << 25), fpa.EUNSUPPORTED),
])
def test_validate(kw, code):
    assert validate_rope(_desc(**kw)) == code


def test_wrong_enums_and_null():
    lib = fpa.load_library()
    assert lib.rope_validate(None) == fpa.EINVAL
    for field, value in (("dtype", 7), ("qkv_order", 2), ("pairs", 2), ("scaling", 3), ("scaling", -1)):
        d = _desc()
        setattr(d, field, value)
        assert validate_rope(d) == fpa.EINVAL, field
    assert lib.rope_create(ctypes.byref(_desc()), None) == fpa.EINVAL
    assert lib.rope_destroy(None) == fpa.OK
    assert lib.rope_split(*[None] * 7) == fpa.EINVAL and lib.rope_rotate(*[None] * 7) == fpa.EINVAL


def test_python_refusals():
    for kw in (dict(dtype=torch.float16), dict(pairs="thirds"), dict(scaling="more"), dict(qkv_order="mixed")):
        with pytest.raises(KeyError):
            _desc(**kw)
    with pytest.raises(fpa.FusedProjError):
        Rope(2, 5, 8, 20)
