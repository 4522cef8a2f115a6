"""Compiles the attention kernels to gfx950 assembly and checks what the compiler does not see to around their inline
direct-to-LDS loads (CPU only: hipcc cross-compiles): the wait states in front of them, and the wait for the zeros that
the same LDS was filled with."""
import os
import re
import shutil

import pytest

from ff_input_projection_amd import build as fpbuild
from test_isa_hazards import HIPCC, _finish_asm, _sgprs, _start_asm, _valu_sgpr_defs

pytestmark = pytest.mark.skipif(shutil.which(HIPCC) is None and not os.path.exists(HIPCC), reason="hipcc not available")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{name: [(instruction, inside inline asm)]} of the attention kernels."""
    d = tmp_path_factory.mktemp("isa")
    outs = [(os.path.join(fpbuild.CSRC, f + ".hip"), os.path.join(d, f + ".s")) for f in ("prompt_attention", "prompt_attention_bwd")]
    procs = [(_start_asm(src, out, 0), out) for src, out in outs]
    found = {}
    for asm in [_finish_asm(p, out) for p, out in procs]:
        for name in re.findall(r"^(_Z\S*attention_(?:kernel|dq_kernel|dkv_kernel)\S*):", asm, re.M):
            a = asm.index("\n" + name + ":")
            insts, in_asm = [], False
            for line in asm[a:asm.index(".Lfunc_end", a)].split("\n"):
                t = line.strip()
                if t.startswith(";;#ASM"):
                    in_asm = t.startswith(";;#ASMSTART")
                elif line.startswith("\t") and t and not t.startswith((".", ";")):
                    insts.append((t, in_asm))
            found[name] = insts
    return found


def test_direct_loads_have_their_wait_states(kernels):
    """5 after a VALU write of an SGPR that the load reads, 1 after a write of M0."""
    checked, problems = 0, []
    for name, insts in kernels.items():
        for i, (t, inside) in enumerate(insts):
            if not inside or not t.startswith("global_load_lds"):
                continue
            checked += 1
            reads, waits, k = _sgprs(t), 0, i - 1
            while k >= 0 and waits < 5:
                p = insts[k][0]
                if p.startswith("s_nop"):
                    waits += int(p.split()[1], 0) + 1
                    k -= 1
                    continue
                if _valu_sgpr_defs(p) & reads:
                    problems.append(f"{name}: '{p}' then '{t}' after {waits} wait states")
                if waits < 1 and re.match(r"s_\w+\s+m0,", p):
                    problems.append(f"{name}: '{p}' then '{t}' with no wait state")
                waits += 1
                k -= 1
    assert checked > 1000, "no direct-to-LDS loads found"
    assert not problems, "\n".join(problems[:20])


def test_zeros_land_before_the_tiles(kernels):
    """Heads narrower than their kernel: the tiles are filled with zeros, and the direct loads that follow write the same LDS
    by another path. A barrier of a workgroup of one wave compiles to nothing, so the kernel has to wait by itself."""
    checked, problems = 0, []
    for name, insts in kernels.items():
        m = re.search(r"attention_(?:dq_|dkv_)?kernelILi\d+ELb(\d)E", name)
        if not int(m.group(1)):
            continue
        first = next(i for i, (t, inside) in enumerate(insts) if inside and t.startswith("global_load_lds"))
        fill = [i for i, (t, _) in enumerate(insts[:first]) if t.startswith("ds_write")]
        assert fill, f"{name}: no zeros"
        checked += 1
        if not any(inside and re.match(r"s_waitcnt.*lgkmcnt\(0\)", t) for t, inside in insts[fill[-1]:first]):
            problems.append(name)
    assert checked >= 50, "no kernels of narrower heads found"
    assert not problems, "\n".join(problems)
