"""Properties of the compiled gfx950 code, checked on the AMD assembly of this
repository's own kernels (CPU only), for every translation unit:

* No vector instruction within two wait states of a store of more than 8 bytes
  writes the store's data registers: the store may still be reading them.  The
  compiler keeps that distance for its own stores, not for one written in
  assembly, and row indexes once replaced outputs that way.
and for the fused kernels' units, what the plain kernels are held to:
* no spills to scratch memory, no packed FP32 operations, no scalar-memory
  writes;
* on any path through the branches, the few-token kernel issues no
  direct-to-LDS copy while an LDS read may be outstanding, and no kernel issues
  one between a barrier that was reached with a read outstanding and the next.
  (LDS instructions keep their order among the waves, copies do not keep it
  with them.)
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


def _kernel_blocks(text):
    """(mangled name, [(label, code lines)] in layout order) of every kernel."""
    name, blocks = None, []
    for line in text.splitlines():
        m = re.match(r"^(_Z\w+):", line)
        label = re.match(r"^(\.LBB\w+):", line)
        if m:
            name, blocks = m.group(1), [("", [])]
        elif name and line.startswith(".Lfunc_end"):
            yield name, blocks
            name = None
        elif name and label:
            blocks.append((label.group(1), []))
        elif name:
            blocks[-1][1].extend(_code_lines(line))


_COPY = r"buffer_load_dword(x4)? .* lds$"


def _outstanding_reads(blocks, few):
    """(barriers, direct-to-LDS copies, lines that break the rule): a copy must not overtake an LDS read that a path
    may have left outstanding at the barrier before it, nor, in the few-token kernel (`few`), one of its own wave."""
    at = {label: i for i, (label, _) in enumerate(blocks)}
    bad, open_barriers = [], []

    def walk(start, state, step):
        """Follows every path from (block, line): state = step(state, line, place), None ends a path."""
        seen, todo = set(), [(start, state)]
        while todo:
            (i, k), state = todo.pop()
            if k == 0:
                if (i, state) in seen:
                    continue
                seen.add((i, state))
            for k in range(k, len(blocks[i][1])):
                s = blocks[i][1][k]
                op = s.split()[0]
                state = step(state, s, (i, k))
                if state is None or op == "s_endpgm":
                    break
                if op == "s_branch" or op.startswith("s_cbranch"):
                    todo.append(((at[s.split()[1]], 0), state))
                    if op == "s_branch":
                        break
            else:
                todo.append(((i + 1, 0), state))

    def reads(pending, s, place):
        if s.startswith("ds_read"):
            return True
        if s.startswith("s_waitcnt") and "lgkmcnt(0)" in s:
            return False
        if pending and s == "s_barrier":
            open_barriers.append(place)
        if pending and few and re.match(_COPY, s):
            bad.append(s)
        return pending

    def copies(state, s, place):
        if re.match(_COPY, s):
            bad.append(s)
        return None if s == "s_barrier" else state

    walk((0, 0), False, reads)
    for i, k in set(open_barriers):
        walk((i, k + 1), True, copies)
    lines = [s for _, body in blocks for s in body]
    return sum(s == "s_barrier" for s in lines), sum(bool(re.match(_COPY, s)) for s in lines), bad


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
    for name, blocks in _kernel_blocks(text):
        b, c, bad = _outstanding_reads(blocks, "fused_decode_kernel" in name)
        assert not bad, f"{name}: a copy may overtake an LDS read: {bad[0]}"
        barriers, copies = barriers + b, copies + c
    assert copies > 0 and barriers > 0


def test_the_check_follows_the_branches():
    read, wait, barrier, copy = "ds_read_b128 v[0:3], v4", "s_waitcnt lgkmcnt(0)", "s_barrier", "buffer_load_dwordx4 v1, s[0:3], 0 offen lds"
    # laid out after a read, but reached from behind the wait only
    moved = [("", [read, "s_branch .L2"]), (".L1", [barrier, copy, "s_endpgm"]), (".L2", [wait, "s_branch .L1"])]
    assert _outstanding_reads(moved, True) == (1, 1, [])
    loop = [("", []), (".L1", [barrier, copy, wait, read, "s_cbranch_scc1 .L1"]), (".L2", [wait, "s_endpgm"])]
    assert _outstanding_reads(loop, False)[2] == [copy]
    assert _outstanding_reads([("", [read, "s_waitcnt lgkmcnt(1)", barrier, copy, "s_endpgm"])], False)[2] == [copy]
    assert _outstanding_reads([("", [read, wait, barrier, copy, "s_endpgm"])], False)[2] == []
    # at the end, nothing is copied any more
    assert _outstanding_reads([("", [read, barrier, "ds_write_b32 v0, v1", "s_endpgm"])], False)[2] == []
    assert _outstanding_reads([("", [read, copy, "s_endpgm"])], True)[2] == [copy]
