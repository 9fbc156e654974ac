"""Static race check of the operators' LDS rings (no GPU).

The rules of ``test_lds_ring`` (what may land, be read and be overwritten when)
over models written from these kernels' source order:
* the persistent 256 x 256 kernel, whose ring is the product's own, with up to
  four rounds of its results through two slots; its K loop in the built code
  objects must issue the model's schedule, for every operation that has one;
* 256 x 128 and 128 x 128 tiles: three stages, twelve and eight loads a step and
  wave;
* 64 x 64 tiles: four stages, each filled after the barrier that frees it;
* few rows of the gated layer: a ring to a wave, where the wave's own wait takes
  the barrier's place;
* the 4-bit product of many rows: x and codes in three stages, scales in two.
The waits in front of the built kernels' barriers are read back too.
"""
from __future__ import annotations

import re

import pytest

import _isa
import test_lds_ring as ring
from dense_fp16_gemm_04_amd import build, operators

SYMBOL = re.compile(r"^[0-9a-f]+ <(\S+)>:")


def kernels(asm: str) -> dict:
    """Kernel symbol -> its instructions' text."""
    out, cur = {}, None
    for l in asm.splitlines():
        m = SYMBOL.match(l)
        if m:
            cur = out.setdefault(m.group(1), [])
        elif cur is not None and l.strip():
            cur.append(l.split("//")[0].strip())
    return out


def barriers(lines) -> list:
    """The counters that the wait in front of each barrier waits for."""
    out, wait = [], ""
    for l in lines:
        if l.startswith("s_waitcnt"):
            wait = l[len("s_waitcnt"):].strip()
        elif l.startswith("s_barrier"):
            out.append(wait)
    return out


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    asm = {n: _isa.disassemble(operators.library_path(n), tmp_path_factory.mktemp(n)) for n in build.OPERATORS}
    return asm, {n: kernels(a) for n, a in asm.items()}


# ------------------------------------------------- 256 x 256, persistent --

def persistent(nk, tiles, rounds):
    """The product's program with `rounds` rounds of results through two slots."""
    ev = ring.ring_program(nk, tiles)
    out, i, done = [], 0, None
    while i < len(ev):
        if ev[i][0] == "write" and ev[i][2] != done:  # (its two rounds, up to their last barrier)
            done = ev[i][2]
            end = max(k for k, e in enumerate(ev) if len(e) > 2 and e[2] == done) + 2  # and the barrier after
            (s0, s1) = (e[1] for e in ev[i:i + 2])
            for _ in range(rounds):
                out += [("write", s0, done), ("write", s1, done), ("bar", 63), ("read", s0, done), ("read", s1, done),
                        ("bar", 63)]
            i = end
        else:
            out.append(ev[i])
            i += 1
    return out


@pytest.mark.parametrize("rounds", [1, 2, 4])
@pytest.mark.parametrize("nk", [3, 4, 5, 6, 7, 8, 9, 12, 17, 128])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4])
def test_persistent_ring(nk, tiles, rounds):
    ev = persistent(nk, tiles, rounds)
    if rounds == 2:
        assert ev == ring.ring_program(nk, tiles)
    assert ring.races(ev) == []


def persistent_symbols(code):
    return [(n, s) for n, ks in code[1].items() for s in ks if "nt_persist" in s]


def test_persistent_loops_issue_the_model_schedule(code, monkeypatch, tmp_path):
    found = persistent_symbols(code)
    # gated forward and its products in two types, S, X' and two results
    assert len(found) >= 8
    for name, symbol in found:
        monkeypatch.setattr(ring, "LEAN_SYMBOL", (symbol,))
        monkeypatch.setattr(ring._isa, "disassemble", lambda lib, tmp, name=name: code[0][name])
        ring.test_lean_loop_issues_the_model_schedule(tmp_path)


# --------------------------------------- 256 x 128 and 128 x 128, ordered --

ORDERED = {"ILi256ELi128E": 12, "ILi128ELi128E": 8}  # loads a step and wave


@pytest.mark.parametrize("loads", sorted(ORDERED.values()))
@pytest.mark.parametrize("nk", [1, 2, 3, 4, 5, 6, 7, 16, 129])
def test_ordered_ring(nk, loads):
    ev = ring.stage_program(nk, 3, loads)
    assert ring.races(ev) == []
    if nk >= 2:
        first = next(i for i, e in enumerate(ev) if e[0] == "bar")
        weak = [("bar", e[1] + 1) if e[0] == "bar" and i > first and e[1] > 0 else e for i, e in enumerate(ev)]
        assert any("landed" in m for _, m in ring.races(weak))


def test_ordered_kernels_wait_as_the_model(code):
    count = 0
    for ks in code[1].values():
        for s, lines in ks.items():
            if "nt_ordered" not in s:
                continue
            size = re.search(r"Li(\d+)ELi(\d+)E", s)
            loads = ORDERED["ILi%sELi%sE" % size.groups()]
            got = barriers(lines)
            # the loading waves' way and the others', a general and a whole step each
            assert got.count("vmcnt(%d) lgkmcnt(0)" % (2 * loads)) == 2 and got.count("vmcnt(%d) lgkmcnt(0)" % loads) == 4, s
            assert "vmcnt(0) lgkmcnt(0)" in got, s
            count += 1
    assert count >= 16


# -------------------------------------------------------- 64 x 64 and few --

def filled_after(nk, stages, loads, order=("bar", "load", "read")):
    """Step ks: wait for its loads, fill the stage that step ks - 1 left, read."""
    ev = []
    for st in range(stages - 1):
        ev += [("load", st, ("AB", st))] * loads
    for ks in range(nk):
        for what in order:
            if what == "bar":
                ev.append(("bar", loads * (stages - 2)))
            elif what == "load":
                ev += [("load", (ks + stages - 1) % stages, ("AB", ks + stages - 1))] * loads
            else:
                ev += [("read", ks % stages, ("AB", ks))] * 4
    ev.append(("bar", 0))
    for st in range(stages):
        ev.append(("write", st, ("C",)))
    ev.append(("bar", 0))
    for st in range(stages):
        ev.append(("read", st, ("C",)))
    return ev


# (stages, loads a step and wave): 64 x 64 tiles; few rows by 8 columns, and by
# 16 columns or for up to 32 rows
@pytest.mark.parametrize("stages, loads", [(4, 4), (3, 6)])
@pytest.mark.parametrize("nk", [0, 1, 2, 3, 4, 5, 9, 64])
def test_rings_filled_after_the_wait(nk, stages, loads):
    ev = filled_after(nk, stages, loads)
    assert ring.races(ev) == []
    if nk > stages:
        weak = [("bar", e[1] + 1) if e[0] == "bar" and e[1] > 0 else e for e in ev]
        assert any("landed" in m for _, m in ring.races(weak))
        # loads before the barrier meet the last step's reads
        early = filled_after(nk, stages, loads, ("load", "bar", "read"))
        assert any("still read" in m for _, m in ring.races(early))


def test_kernels_filled_after_the_wait_wait_as_the_model(code):
    tiles = few = 0
    for s, lines in code[1]["gated_nt"].items():
        if "nt_tile" in s:
            assert barriers(lines)[0] == "vmcnt(8) lgkmcnt(0)" and barriers(lines)[1] == "vmcnt(0) lgkmcnt(0)", s
            tiles += 1
        if "gated_few" in s:
            mb, g = (int(v) for v in re.search(r"Li(\d+)ELi(\d+)E", s).groups())
            loads = 2 * mb + 2 * g // 8
            stages = 4 if loads == 4 else 3
            assert loads in (4, 6)
            # one wait of the loop, before that iteration's loads; all loads have
            # landed before the partial sums take their place
            wait = "s_waitcnt vmcnt(%d) lgkmcnt(0)" % ((stages - 2) * loads)
            at = lines.index(wait)
            assert lines.count(wait) == 1
            back = [i for i, l in enumerate(lines) if i > at and l.startswith("s_cbranch")][0]
            body = lines[at:back]
            assert sum(l.startswith("buffer_load_dwordx4") and l.endswith("lds") for l in body) == loads, s
            assert sum(l.startswith("ds_read_b128") for l in body) == 2 * (mb + 2 * g // 16), s
            assert barriers(lines)[0] == "vmcnt(0) lgkmcnt(0)", s
            few += 1
    assert tiles >= 8 and few == 12


# -------------------------------------------------- 4-bit, many rows of x --

def many_rows(blocks, loads_codes, window=2, early=False):
    """One wave of gemm_w4: block b's x and codes in stage b % 3, its scales in
    half b % 2, read from memory a block ahead into registers (which count among
    the loads in flight) and written behind the block's products.  `early`: into
    the block's own half, in front of them."""
    ev = []
    x, w, s = (lambda b: b % 3), (lambda b: 3 + b % 3), (lambda b: 6 + b % 2)

    def load(b):
        ev.extend([("load", w(b), ("w", b))] * loads_codes)
        ev.extend([("load", x(b), ("x", b))] * 2)

    def scales(b):
        ev.append(("load", 8 + b, ("register", b)))

    scales(0)
    load(0)
    load(1)
    ev.append(("write", s(0), ("s", 0)))
    for b in range(blocks):
        ev.append(("bar", window))
        scales(b + 1)
        load(b + 2)
        if early:
            ev.append(("write", s(b), ("s", b + 1)))
        ev.append(("read", x(b), ("x", b)))
        if loads_codes:  # (the other waves read what these have loaded)
            ev.append(("read", w(b), ("w", b)))
        ev.append(("read", s(b), ("s", b)))
        ev.append(("write", s(b + 1), ("s", b + 1)))
    ev.append(("bar", 0))
    for st in range(3):
        ev.append(("write", st, ("sums",)))
    ev.append(("bar", 0))
    for st in range(3):
        ev.append(("read", st, ("sums",)))
    return ev


# (waves that load codes and waves that load x only)
@pytest.mark.parametrize("loads_codes", [0, 1])
@pytest.mark.parametrize("blocks", [0, 1, 2, 3, 4, 7, 32])
def test_many_rows_ring(blocks, loads_codes):
    assert ring.races(many_rows(blocks, loads_codes)) == []
    if blocks > 3:
        # x of the block itself, still in flight
        assert any("landed" in m for _, m in ring.races(many_rows(blocks, loads_codes, window=4 + loads_codes)))
        assert ring.races(many_rows(blocks, loads_codes, early=True)) != []


def test_many_rows_kernels_wait_as_the_model(code):
    found = [lines for s, lines in code[1]["gemv_w4"].items() if "gemm_w4" in s]
    assert len(found) == 10
    for lines in found:
        assert barriers(lines)[:2] == ["vmcnt(2) lgkmcnt(0)", "vmcnt(0) lgkmcnt(0)"]
