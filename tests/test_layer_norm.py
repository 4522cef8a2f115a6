"""Layer norm's descriptor, refusals and exports, without a GPU."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import ff_input_projection_amd as fpa
from ff_input_projection_amd import LayerNorm, make_layer_norm_desc, validate_layer_norm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_exports_what_the_header_declares():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "layer_norm.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b(layer_norm_[a-z_]+)\s*\(", text))
    assert declared == set(fpa.LAYER_NORM_SYMBOLS)
    lib = fpa.load_library()
    for name in declared:
        assert hasattr(lib, name), name


def test_descriptor_layout_matches_c(tmp_path):
    src = ('#include <stdio.h>\n#include <stddef.h>\n#include "layer_norm.h"\n'
           'int main(void){printf("%zu %zu %zu %zu\\n", sizeof(layer_norm_desc), offsetof(layer_norm_desc, channels), '
           'offsetof(layer_norm_desc, x_stride_spatial), offsetof(layer_norm_desc, eps)); return 0;}\n')
    exe = str(tmp_path / "layout")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-x", "c", "-",
                        "-o", exe], input=src, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    vals = list(map(int, subprocess.run([exe], capture_output=True, text=True).stdout.split()))
    D = fpa.LayerNormDesc
    assert vals == [ctypes.sizeof(D), D.channels.offset, D.x_stride_spatial.offset, D.eps.offset]


def _desc(shape=(2, 8, 5), strides=None, layout="tokens_last", dtype=torch.float32, **kw):
    if strides is None:
        strides = torch.empty(shape, device="meta").stride()
    return make_layer_norm_desc(shape, strides, layout, dtype, **kw)


@pytest.mark.parametrize("desc,code", [
    (lambda: _desc(), fpa.OK),
    (lambda: _desc(dtype=torch.bfloat16, shape=(3, 1, 1)), fpa.OK),
    (lambda: _desc((2, 8, 5), (100, 9, 1)), fpa.OK),                               # rows of a wider tensor, odd stride
    (lambda: _desc((2, 8, 5), (0, 5, 1)), fpa.OK),                                 # one slab for every sequence
    (lambda: _desc((2, 8, 5), (80, 10, 2)), fpa.EUNSUPPORTED),                     # every other channel
    (lambda: _desc((2, 3, 32768)), fpa.OK),
    (lambda: _desc((2, 3, 32769)), fpa.EUNSUPPORTED),
    (lambda: _desc((2, 7, 3, 5, 2), layout="channels_first"), fpa.OK),
    (lambda: _desc((2, 7, 3, 5), (105, 15, 1, 3), layout="channels_first"), fpa.EUNSUPPORTED),   # a transposed grid
    (lambda: _desc((2, 40000, 3), layout="channels_first"), fpa.OK),
    (lambda: _desc((0, 8, 5)), fpa.OK),
    (lambda: _desc((2, 0, 5)), fpa.OK),
    (lambda: _desc((2, 8, 0)), fpa.EINVAL),                                        # no channels: no mean
    (lambda: _desc((2, 8, 5), (-40, 5, 1)), fpa.EINVAL),
    (lambda: _desc(eps=-1e-5), fpa.EINVAL),
    (lambda: _desc(eps=float("nan")), fpa.EINVAL),
    (lambda: _desc(eps=float("inf")), fpa.EINVAL),
    (lambda: _desc(eps=0.0), fpa.OK),
    (lambda: _desc((1 << 20, 1 << 12, 8), (0, 0, 1)), fpa.EUNSUPPORTED),           # 2^32 tokens
])
def test_validate(desc, code):
    assert validate_layer_norm(desc()) == code


def test_wrong_enums_and_null():
    assert fpa.load_library().layer_norm_validate(None) == fpa.EINVAL
    for field, value in (("dtype", 7), ("x_layout", 2), ("has_bias", 2), ("n_spatial", 2)):
        d = _desc()
        setattr(d, field, value)
        assert validate_layer_norm(d) == fpa.EINVAL, field
    assert fpa.load_library().layer_norm_create(ctypes.byref(_desc()), None) == fpa.EINVAL
    assert fpa.load_library().layer_norm_destroy(None) == fpa.OK


def test_python_refuses_what_is_no_activation():
    with pytest.raises(ValueError):
        make_layer_norm_desc((2, 8), (8, 1), "tokens_last", torch.float32)
    with pytest.raises(ValueError):
        make_layer_norm_desc((2, 8), (8, 1), "channels_first", torch.float32)
    with pytest.raises(ValueError):
        make_layer_norm_desc((2, 8, 4), (32, 4, 1), "sideways", torch.float32)
    with pytest.raises(KeyError):
        make_layer_norm_desc((2, 8, 4), (32, 4, 1), "tokens_last", torch.float16)
    with pytest.raises(fpa.FusedProjError):
        LayerNorm((2, 8, 5), (80, 10, 2), "tokens_last", torch.float32)


@pytest.mark.parametrize("shape,strides,layout,code", [
    ((1, (1 << 31) - (1 << 23), 1), (0, 0, 1), "tokens_last", fpa.OK),
    ((1, (1 << 31) - (1 << 23) + 1, 1), (0, 0, 1), "tokens_last", fpa.EUNSUPPORTED),
    (((1 << 31) - 1, 1, 1), (0, 0, 1), "channels_first", fpa.EUNSUPPORTED),
    ((0, 1, (1 << 31) - 1), (0, 0, 1), "channels_first", fpa.EUNSUPPORTED),
    ((1, 1 << 29, 1), (0, 0, 1), "channels_first", fpa.OK),
    ((1, (1 << 29) + 1, 1), (0, 0, 1), "channels_first", fpa.EUNSUPPORTED),
])
def test_sizes_that_32_bit_loops_would_pass_are_refused(shape, strides, layout, code):
    assert validate_layer_norm(_desc(shape, strides, layout)) == code
