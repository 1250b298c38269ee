"""Properties of the compiled gfx950 code, checked on the AMD assembly of this
repository's own kernels (CPU only), for every translation unit:

* No vector instruction within two wait states of a store of more than 8 bytes
  writes the store's data registers: the store may still be reading them.  The
  compiler keeps that distance for its own stores, not for one written in
  assembly, and row indexes once replaced outputs that way.
and for the fused kernels' units, what the plain kernels are held to:
* no spills to scratch memory, no packed FP32 operations, no scalar-memory
  writes;
* the few-token kernel issues no direct-to-LDS copy while an LDS read may be
  outstanding, and no kernel reaches a barrier with one outstanding.
"""
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from fp8_gemm_amd import _build
from tests.test_isa_invariants import _code_lines, _kernels

UNITS = [_build.SRC] + _build.FUSED_SRCS


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if shutil.which("hipcc") is None and not os.path.exists(_build.hipcc()):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("isa")

    def compile_one(src):
        dst = out / (os.path.basename(src) + ".s")
        flags = [f for f in _build.HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
        subprocess.run([_build.hipcc()] + flags + ["-S", "--cuda-device-only", src, "-o", str(dst)], check=True,
                       capture_output=True)
        return dst.read_text()

    with ThreadPoolExecutor(len(UNITS)) as pool:
        return dict(zip(UNITS, pool.map(compile_one, UNITS)))


def _registers(operand):
    """The register numbers of v7, v[4:7] or a[0:3] (AGPRs as negative numbers)."""
    m = re.match(r"([va])\[(\d+):(\d+)\]$", operand) or re.match(r"([va])((\d+))$", operand)
    if not m:
        return set()
    numbers = range(int(m.group(2)), int(m.group(3)) + 1)
    return {n if m.group(1) == "v" else -1 - n for n in numbers}


def _overwritten_stores(body):
    """(number of wide stores, those whose data a following vector instruction overwrites too early)."""
    stores, bad = 0, []
    for i, this in enumerate(body):
        op, _, rest = this.partition(" ")
        if not re.match(r"(global|buffer|flat)_store_dwordx[34]$", op):
            continue
        args = [a.strip() for a in rest.split(",")]
        data = _registers(args[0 if op.startswith("buffer") else 1])
        assert data, this
        stores += 1
        states = 0
        for after in body[i + 1:]:
            nop, _, dest = after.partition(" ")
            if nop.startswith("v_") and not nop.startswith("v_cmp") and _registers(dest.split(",")[0].strip()) & data:
                bad.append(f"{this} / {after}")
            states += int(dest) + 1 if nop == "s_nop" else 1
            if states >= 2 or nop in ("s_branch", "s_endpgm"):
                break
    return stores, bad


def test_wide_store_data_not_overwritten(asm):
    total = 0
    for unit, text in asm.items():
        for name, body in _kernels(text):
            stores, bad = _overwritten_stores(body)
            total += stores
            assert not bad, f"{name}: {bad[0]}"
    assert total > 0


def test_the_check_sees_an_early_write():
    store = "global_store_dwordx4 v[134:135], v[130:133], off sc1"
    write = "v_lshl_or_b32 v130, s22, 4, v196"
    assert _overwritten_stores([store, "s_or_b64 exec, exec, s[12:13]", write])[1]
    assert not _overwritten_stores([store, "s_nop 1", write])[1]


@pytest.mark.parametrize("unit", _build.FUSED_SRCS, ids=os.path.basename)
def test_fused_units_hold_the_plain_kernels_rules(asm, unit):
    text = asm[unit]
    sizes = [int(v) for v in re.findall(r"\.private_segment_fixed_size:\s*(\d+)", text)]
    assert sizes and max(sizes) == 0
    for s in _code_lines(text):
        op = s.split()[0]
        assert not re.match(r"v_pk_(add|mul|fma)_f32", op), s
        assert not re.match(r"s_(buffer_)?(store|atomic)|s_dcache_(wb|discard)", op), s
    copies = barriers = 0
    for name, body in _kernels(text):
        pending = False
        for s in body:
            op = s.split()[0]
            if op.startswith("ds_read"):
                pending = True
            elif op == "s_waitcnt" and re.search(r"lgkmcnt\(0\)", s):
                pending = False
            elif op == "s_barrier":
                assert not pending, f"{name}: barrier with an LDS read outstanding"
                barriers += 1
            elif "fused_decode_kernel" in name and re.match(r"buffer_load_dword(x4)? ", s) and s.endswith(" lds"):
                assert not pending, f"{name}: LDS copy issued with an LDS read outstanding: {s}"
                copies += 1
    assert copies > 0 and barriers > 0
