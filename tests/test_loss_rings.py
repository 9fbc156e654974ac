"""Static race check of the LDS rings and images of the loss over a vocabulary (no GPU).

Its products run on the rings of ``test_operator_rings``; what is its own:
* the persistent kernel's epilogue with no results through LDS (the loss, sums
  kept in 32 bits), and with four rounds of two images (dl both ways round);
* in the built code the persistent loops issue the model's schedule, and the
  ordered kernels wait as theirs, those that read W as it lies too;
* W's rows as they lie in LDS.
"""
from __future__ import annotations

import re

import pytest

import _isa
import test_lds_ring as ring
import test_operator_rings as rings
from dense_fp16_gemm_04_amd import operators

NAME = "linear_cross_entropy"


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    asm = _isa.disassemble(operators.library_path(NAME), tmp_path_factory.mktemp(NAME))
    return asm, rings.kernels(asm)


def without_results(nk, tiles):
    """The ring's program with an epilogue that uses no LDS: what is left of it are its barriers."""
    return [e for e in rings.persistent(nk, tiles, 1) if not (e[0] in ("write", "read") and len(e) > 2 and str(e[2][0]) == "C")]


@pytest.mark.parametrize("nk", [3, 4, 5, 6, 7, 8, 9, 12, 17, 33, 128])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 7])
def test_persistent_ring(nk, tiles):
    assert ring.races(rings.persistent(nk, tiles, 4)) == []
    assert ring.races(without_results(nk, tiles)) == []


def test_persistent_loops_issue_the_model_schedule(code, monkeypatch, tmp_path):
    found = [s for s in code[1] if "nt_persist" in s]
    # in two types: the loss, dl, the sums, dX in four forms, dW in two
    assert len(found) == 18
    for symbol in found:
        monkeypatch.setattr(ring, "LEAN_SYMBOL", (symbol,))
        monkeypatch.setattr(ring._isa, "disassemble", lambda lib, tmp: code[0])
        ring.test_lean_loop_issues_the_model_schedule(tmp_path)


def test_ordered_kernels_wait_as_the_model(code):
    found = {s: lines for s, lines in code[1].items() if "nt_ordered" in s}
    # each as two tiles in two types: the loss, dl, the sums and dX in four forms, both
    # on a transposed W and on W as it lies, dW in two
    assert len(found) == 56
    turned = [s for s, lines in found.items() if any(l.startswith("ds_read_b64_tr_b16") for l in lines)]
    assert len(turned) == 20 and all("AddOp" in s or "DxOp" in s for s in turned)
    for s, lines in found.items():
        size = re.search(r"Li(\d+)ELi(\d+)E", s)
        loads = rings.ORDERED["ILi%sELi%sE" % size.groups()]
        got = rings.barriers(lines)
        assert got.count("vmcnt(%d) lgkmcnt(0)" % (2 * loads)) == 2 and got.count("vmcnt(%d) lgkmcnt(0)" % loads) == 4, s
        assert "vmcnt(0) lgkmcnt(0)" in got, s


def test_accumulators_are_read_after_their_products(code):
    """Between the last product and the first read of a 256 x 256 tile's
    accumulators by name (which the compiler's hazard checks do not see) lie
    the waits that the longest product needs: 24 cycles at least."""
    checked = 0
    for s, lines in code[1].items():
        if "nt_persist" not in s:
            continue
        last = None
        for i, l in enumerate(lines):
            if l.startswith("v_mfma"):
                last, idle = i, 0
            elif last is not None and l.startswith("s_nop"):
                idle += int(l.split()[1], 0) + 1
            elif last is not None and l.startswith("v_accvgpr_read"):
                assert idle >= 24, (s, i)
                checked += 1
                last = None
    assert checked >= 18


def turned_swizzle(k, chunk):
    return chunk ^ ((k & 3) << 1) ^ (((k >> 3) & 1) << 3)


def test_rows_of_w_in_lds():
    """Rows of 128 columns, 64 of them: each of the loads' 16-byte pieces has a place of its
    own, a fragment's reads find their columns, and those of a wave, 512 bytes, fall
    on all 64 banks evenly."""
    places = {}
    for wave in range(4):
        for load in range(4):
            for lane in range(64):
                k = wave * 16 + load * 4 + lane // 16
                places[(wave * 4 + load) * 1024 + lane * 16] = (k, turned_swizzle(k, lane % 16))
    assert sorted(places) == list(range(0, 64 * 256, 16)) and len(set(places.values())) == 64 * 16
    for first in range(0, 128, 16):  # of a block's 16 columns
        for step in (0, 32):
            for half in (0, 4):
                banks = [0] * 64
                for lane in range(64):
                    r, k = lane % 16, lane // 16 * 8 + lane % 16 // 4
                    at = k * 256 + turned_swizzle(k, first // 8 + r % 4 // 2) * 16 + r % 2 * 8 + (step + half) * 256
                    k += step + half
                    assert places[at // 16 * 16] == (k, (first + r % 4 * 4) // 8) and at % 16 == (first + r % 4 * 4) % 8 * 2
                    for b in range(2):
                        banks[at // 4 % 64 + b] += 1
                assert banks == [2] * 64
