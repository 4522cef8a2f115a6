"""The key/value cache's descriptor, refusals and exports, without a GPU."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import ff_input_projection_amd as fpa
from ff_input_projection_amd import KVCache, make_kv_cache_desc, validate_kv_cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_exports_what_the_header_declares():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kv_cache.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b(kv_cache_[a-z_]+)\s*\(", text))
    assert declared == set(fpa.KV_CACHE_SYMBOLS)
    lib = fpa.load_library()
    for name in declared:
        assert hasattr(lib, name), name


def test_descriptor_layout_matches_c(tmp_path):
    src = ('#include <stdio.h>\n#include <stddef.h>\n#include "kv_cache.h"\n'
           'int main(void){printf("%zu %zu %zu %zu %zu\\n", sizeof(kv_cache_desc), offsetof(kv_cache_desc, tokens), '
           'offsetof(kv_cache_desc, max_pages), offsetof(kv_cache_desc, sm_scale), sizeof(kv_cache_storage)); return 0;}\n')
    exe = str(tmp_path / "layout")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-x", "c", "-",
                        "-o", exe], input=src, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    vals = list(map(int, subprocess.run([exe], capture_output=True, text=True).stdout.split()))
    D = fpa.KVCacheDesc
    assert vals == [ctypes.sizeof(D), D.tokens.offset, D.max_pages.offset, D.sm_scale.offset,
                    ctypes.sizeof(fpa.KVCacheStorage)]


def _desc(batch=2, tokens=1, n_heads=8, head_dim=64, **kw):
    return make_kv_cache_desc(batch, tokens, n_heads, head_dim, **{**dict(n_pages=5, max_pages=2), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(), fpa.OK), (dict(bits=8), fpa.OK), (dict(batch=0), fpa.OK), (dict(n_kv_heads=2), fpa.OK),
    (dict(head_dim=24), fpa.OK), (dict(head_dim=512), fpa.OK), (dict(page_size=48), fpa.OK), (dict(sm_scale=0.5), fpa.OK),
    (dict(bits=3), fpa.EINVAL), (dict(batch=-1), fpa.EINVAL), (dict(tokens=0), fpa.EINVAL), (dict(n_heads=0), fpa.EINVAL),
    (dict(n_kv_heads=3), fpa.EINVAL), (dict(n_kv_heads=-1), fpa.EINVAL), (dict(head_dim=0), fpa.EINVAL),
    (dict(n_pages=0), fpa.EINVAL), (dict(max_pages=0), fpa.EINVAL), (dict(page_size=0), fpa.EINVAL),
    (dict(sm_scale=-1.0), fpa.EINVAL), (dict(sm_scale=float("inf")), fpa.EINVAL), (dict(sm_scale=float("nan")), fpa.EINVAL),
    (dict(dtype=torch.float32), fpa.EUNSUPPORTED), (dict(head_dim=20), fpa.EUNSUPPORTED),
    (dict(head_dim=520), fpa.EUNSUPPORTED), (dict(page_size=24), fpa.EUNSUPPORTED),
    (dict(page_size=65552), fpa.EUNSUPPORTED), (dict(max_pages=1 << 26, page_size=64), fpa.EUNSUPPORTED),
    (dict(max_pages=1 << 24, page_size=64), fpa.EUNSUPPORTED), (dict(max_pages=(1 << 24) - 1, page_size=64), fpa.OK),
    (dict(batch=1 << 14, tokens=1 << 13, head_dim=512), fpa.EUNSUPPORTED), (dict(tokens=1 << 27), fpa.EUNSUPPORTED),
    (dict(max_pages=1 << 62), fpa.EUNSUPPORTED), (dict(batch=1 << 20, tokens=1 << 12), fpa.EUNSUPPORTED),
    (dict(n_pages=(1 << 31) - 1, page_size=65536, n_heads=1 << 20), fpa.EUNSUPPORTED),
])
def test_validate(kw, code):
    assert validate_kv_cache(_desc(**kw)) == code


def test_null_arguments():
    lib = fpa.load_library()
    assert lib.kv_cache_validate(None) == fpa.EINVAL
    assert lib.kv_cache_create(ctypes.byref(_desc()), None) == fpa.EINVAL
    assert lib.kv_cache_destroy(None) == fpa.OK
    n = ctypes.c_size_t()
    assert lib.kv_cache_storage_bytes(None, ctypes.byref(n), ctypes.byref(n)) == fpa.EINVAL
    assert lib.kv_cache_attend_workspace_size(None, ctypes.byref(n)) == fpa.EINVAL


def test_python_refusals():
    with pytest.raises(KeyError):
        _desc(dtype=torch.float16)
    with pytest.raises(fpa.FusedProjError):
        KVCache(2, 1, 8, 20, n_pages=5, max_pages=2)


def test_validate_bounds_the_logits_factor():
    """sm_scale log2(e), what the kernels multiply by, has to be an fp32 number."""
    assert validate_kv_cache(_desc(sm_scale=2.3e38)) == fpa.OK
    assert validate_kv_cache(_desc(sm_scale=2.4e38)) == fpa.EINVAL
