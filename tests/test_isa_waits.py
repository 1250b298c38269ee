"""Wait states that the hardware leaves to the program and that the compiler
keeps for its own instructions but not around inline assembly, checked on the
AMD assembly of this repository's own kernels (CPU only), in code order:

* one between a scalar write of M0 and a load that takes its LDS address from
  M0 (`buffer_load ... lds`);
* five between a vector instruction that writes a scalar register (a lane read
  into a descriptor word) and a buffer or global access that reads it.

Every instruction between counts as one, `s_nop N` as N + 1.
"""
import os
import re

import pytest

from tests.test_isa_fused import UNITS, asm  # noqa: F401 (asm: fixture)
from tests.test_isa_invariants import _kernels

_ACCESS = re.compile(r"(buffer|global|flat)_(load|store|atomic)")


def _scalars(operand):
    """The scalar registers of s7 or s[4:7]."""
    m = re.match(r"s\[(\d+):(\d+)\]$", operand) or re.match(r"s((\d+))$", operand)
    return set(range(int(m.group(1)), int(m.group(2)) + 1)) if m else set()


def _states(line):
    op, _, rest = line.partition(" ")
    return int(rest) + 1 if op == "s_nop" else 1


def _too_early(body):
    """(accesses, loads to LDS, the pairs that break a rule)."""
    accesses = loads = 0
    bad = []
    for i, this in enumerate(body):
        if not _ACCESS.match(this):
            continue
        accesses += 1
        to_lds = this.endswith(" lds")
        loads += to_lds
        reads = set().union(*(_scalars(word) for word in re.split(r"[ ,]+", this)[1:]))
        states = 0
        for before in reversed(body[max(0, i - 5):i]):
            op, _, rest = before.partition(" ")
            dest = rest.split(",")[0].strip()
            if (to_lds and states < 1 and op.startswith("s_") and dest == "m0") or \
                    (op.startswith("v_") and states < 5 and _scalars(dest) & reads):
                bad.append(f"{before} / {this}")
            states += _states(before)
            if states >= 5:
                break
    return accesses, loads, bad


@pytest.mark.parametrize("unit", UNITS, ids=os.path.basename)
def test_accesses_wait_for_what_they_read(asm, unit):  # noqa: F811
    accesses = loads = 0
    for name, body in _kernels(asm[unit]):
        a, n, bad = _too_early(body)
        assert not bad, f"{name}: {len(bad)}, first {bad[0]}"
        accesses, loads = accesses + a, loads + n
    assert accesses > loads > 0


def test_the_check_sees_early_accesses():
    load = "buffer_load_dwordx4 v1, s[4:7], 0 offen lds"
    assert _too_early(["s_add_i32 m0, s1, 0x400", load])[2]
    assert not _too_early(["s_add_i32 m0, s1, 0x400", "s_nop 0", load])[2]
    assert not _too_early(["s_mov_b32 m0, s1", "v_add_u32_e32 v1, v2, v3", load])[2]
    assert not _too_early(["s_mov_b32 m0, s1", "buffer_load_dwordx4 v1, s[4:7], 0 offen"])[2]
    assert _too_early(["v_readfirstlane_b32 s6, v9", "s_nop 3", load])[2]
    assert not _too_early(["v_readfirstlane_b32 s6, v9", "s_nop 4", load])[2]
    assert not _too_early(["v_readfirstlane_b32 s8, v9", load])[2]
