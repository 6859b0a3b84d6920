"""The product kernels that issue matrix instructions from inline asm keep the
wait states that the compiler cannot see there.

A vector write of a register needs two wait states before a matrix instruction
reads it, and a matrix instruction's result needs up to 19 before anything but
another matrix instruction reads it.  The compiler inserts them around its own
matrix instructions only; here the operands come from LDS (which the compiler
does wait for) and the sums are zeroed long before and read after an explicit
wait, so no listing may hold either pattern.  Compiles the source to AMD
assembly on the CPU, with the library's own flags."""
import os
import re

import pytest

from test_isa import CSRC, _asm, _bodies

READ_AFTER = 19
WRITE_BEFORE = 2


def _regs(tok):
    m = re.match(r"([va])\[(\d+):(\d+)\]$", tok) or re.match(r"([va])(\d+)$", tok)
    if not m:
        return set()
    lo, hi = int(m.group(2)), int(m.group(m.lastindex))
    return {(m.group(1), i) for i in range(lo, hi + 1)}


def _split(ins):
    parts = ins.replace(",", " ").split()
    return parts[0], [_regs(p) for p in parts[1:]]


def _states(ins):
    return int(ins.split()[1], 0) + 1 if ins.startswith("s_nop") else 1


def _written(op, regs):
    """Registers that a vector instruction (no matrix one) writes."""
    if not op.startswith("v_") or op.startswith(("v_mfma", "v_cmp", "v_readlane", "v_readfirstlane")) or not regs:
        return set()
    return regs[0] | (regs[1] if op.startswith("v_swap") else set())


def _read(op, regs):
    """Registers that anything but a matrix instruction reads."""
    if op.startswith("v_mfma"):
        return set()
    first = 0 if op.startswith(("ds_write", "global_store", "buffer_store", "v_cmp", "v_swap")) else 1
    return set().union(*regs[first:]) if regs[first:] else set()


def matrix_hazards(text, kernels):
    """(kernel, first instruction, second) of every pair that is too close, in
    the order of the listing."""
    hits = []
    for name, body in _bodies(text):
        if not re.search(kernels, name):
            continue
        for i, ins in enumerate(body):
            op, regs = _split(ins)
            if not op.startswith("v_mfma"):
                continue
            operands = set().union(*regs[1:])
            waited = 0
            for prev in reversed(body[:i]):
                if waited >= WRITE_BEFORE:
                    break
                if _written(*_split(prev)) & operands:
                    hits.append((name, prev, ins))
                    break
                waited += _states(prev)
            waited = 0
            for nxt in body[i + 1:]:
                if waited >= READ_AFTER:
                    break
                if _read(*_split(nxt)) & regs[0]:
                    hits.append((name, ins, nxt))
                    break
                waited += _states(nxt)
    return hits


def test_detector():
    def hits(*body):
        return matrix_hazards("_Z1kv:\n" + "".join("\t%s\n" % b for b in body) + ".Lfunc_end0:\n", "_Z1kv")
    m = "v_mfma_i32_16x16x64_i8 a[0:3], v[4:7], v[8:11], a[0:3]"
    assert hits("ds_read_b128 v[4:7], v0", "s_waitcnt lgkmcnt(0)", m) == []
    assert len(hits("v_mov_b32 v5, v0", m)) == 1                               # an operand
    assert len(hits("v_mov_b32 v5, v0", "s_nop 0", m)) == 1
    assert hits("v_mov_b32 v5, v0", "s_nop 1", m) == []
    assert hits("v_mov_b32 v5, v0", "v_mov_b32 v20, v0", "v_mov_b32 v21, v0", m) == []
    assert len(hits("v_accvgpr_write_b32 a2, 0", "v_mov_b32 v20, v0", m)) == 1   # a sum
    assert hits("v_mov_b32 v12, v0", m) == []
    assert len(hits(m, "s_nop 15", "v_accvgpr_read_b32 v20, a1")) == 1
    assert hits(m, "s_nop 15", "s_nop 7", "v_accvgpr_read_b32 v20, a1") == []
    assert len(hits(m, "ds_write_b128 v0, a[0:3]")) == 1
    assert hits(m, m) == []                                                    # a chain of sums has its own rule


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    return _asm(os.path.join(CSRC, "tq_epilogue.hip"), str(tmp_path_factory.mktemp("isa")))


def test_products_from_asm_wait(listing):
    names = [n for n, body in _bodies(listing) if "k_epi_ring" in n and any(b.startswith("v_mfma") for b in body)]
    assert len(names) == 12                  # three types, four tiles and rings
    hits = matrix_hazards(listing, "k_epi_ring")
    assert not hits, "\n".join("%s\n    %s\n    %s" % h for h in hits[:10])
