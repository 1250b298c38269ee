"""Properties of the compiled gfx950 code of the experts' and integer kernels that
tests/test_isa_fused.py does not name (CPU only; it holds both units to the plain
kernels' rules):

* the few-token kernel over ragged groups, whose waves refill their own ring slots
  without a barrier, issues no direct-to-LDS copy while an LDS read may be
  outstanding, on any path;
* the persistent kernels read their sums only after the wait that the pins hide
  from the compiler: the last matrix instruction before an accumulator is read
  is at least 20 wait states back;
* no build copies sums between the register files in its main loop.
"""
import os
import re

import pytest

from fp8_gemm_amd import _build
from tests.test_isa_fused import _kernel_blocks, _outstanding_reads, _registers, asm  # noqa: F401 (asm: fixture)

UNITS = _build.EXPERTS_SRCS


@pytest.mark.parametrize("unit", UNITS, ids=os.path.basename)
def test_few_token_copies_wait_for_reads(asm, unit):  # noqa: F811
    kernels = copies = 0
    for name, blocks in _kernel_blocks(asm[unit]):
        if "ragged_decode_kernel" not in name:
            continue
        kernels += 1
        _, c, bad = _outstanding_reads(blocks, True)
        assert not bad, f"{name}: a copy may overtake an LDS read: {bad[0]}"
        copies += c
    assert kernels == 9 and copies > 0


def _states(line):
    op, _, rest = line.partition(" ")
    return int(rest) + 1 if op == "s_nop" else 1


def _early_reads(body):
    """(matrix instructions, reads of an accumulator by anything else within 20 wait states of its writing, in code order)."""
    count, bad, written = 0, [], {}
    clock = 0
    for s in body:
        op, _, rest = s.partition(" ")
        args = [a.strip() for a in rest.split(",")]
        if op.startswith("v_mfma"):
            count += 1
            for r in _registers(args[0]):
                written[r] = clock
        else:
            reads = set().union(*(_registers(a) for a in (args if "store" in op or op.startswith("ds_write") else args[1:])), set())
            bad += [s for r in reads if r < 0 and clock - written.get(r, -100) < 20]
        clock += _states(s)
    return count, bad


@pytest.mark.parametrize("unit", UNITS, ids=os.path.basename)
def test_sums_are_read_after_their_wait(asm, unit):  # noqa: F811
    kernels = 0
    for name, blocks in _kernel_blocks(asm[unit]):
        if "tile_kernel" not in name:
            continue
        count, bad = _early_reads([s for _, body in blocks for s in body])
        assert count and not bad, f"{name}: {bad[:1]}"
        kernels += 1
    assert kernels >= 15


def test_the_check_sees_an_early_read():
    mfma, read = "v_mfma_i32_16x16x64_i8 a[0:3], v[0:3], v[4:7], a[0:3]", "v_accvgpr_read_b32 v8, a2"
    assert _early_reads([mfma, "s_nop 15", read])[1] == [read]
    assert _early_reads([mfma, "s_nop 15", "s_nop 7", read])[1] == []
    assert _early_reads([mfma, "ds_write_b128 v1, a[0:3]"])[1]


@pytest.mark.parametrize("unit", UNITS, ids=os.path.basename)
def test_main_loops_keep_their_sums(asm, unit):  # noqa: F811
    loops = 0
    for name, blocks in _kernel_blocks(asm[unit]):
        if "tile_kernel" not in name:
            continue
        for label, body in blocks:
            mfma = sum(s.startswith("v_mfma") for s in body)
            if mfma >= 8:
                loops += 1
                # (the loop's last block may go on into the clearing of the next tile's sums)
                back = next((i for i, s in enumerate(body) if s.startswith("s_cbranch") and s.split()[1] == label), len(body))
                assert not [s for s in body[:back] if s.startswith("v_accvgpr")], f"{name} {label}"
    assert loops >= 15
