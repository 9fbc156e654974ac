"""Newton-Schulz at the ends of G's range: norms whose inverse 32 bits cannot
hold, zero matrices, infinities, rows and columns far below the others, and
polynomials that grow and shrink."""
from __future__ import annotations

import pytest
import torch

import _ns
import _operators as plain
import dense_fp16_gemm_04_amd as fw
from test_operators import DEV, _built, normal, ns_close  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(33, 50), (70, 200), (300, 90), (2, 40, 64)]


@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("power", [-146, -140, -130, -100, 100, 120])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_ns_of_tiny_and_huge_entries(shape, power, t):
    # (entries of at most 5, down to subnormal ones)
    g = (normal(*shape, seed=3).double() * 2.0 ** power).to({"fp32": torch.float32, "bf16": torch.bfloat16}[t])
    if float(g.double().abs().max()) == 0:
        assert power < -133 and t == "bf16"
        return
    for steps in (0, 5):
        ns_close(fw.orthogonalize_ns(g, steps=steps, eps=0.0), g, steps=steps, eps=0.0)


def test_ns_of_the_largest_entries():
    """Every entry the type's largest: the factor to X is below 32 bits' normal range."""
    for shape in ((40, 60), (200, 3000)):
        signs = normal(*shape, seed=4).sign()
        g = signs * torch.finfo(torch.float32).max
        for steps in (0, 3):
            ns_close(fw.orthogonalize_ns(g, steps=steps), g, steps=steps)
            assert torch.equal(fw.orthogonalize_ns(g, steps=steps), fw.orthogonalize_ns(signs, steps=steps, eps=0.0))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_ns_of_zero_matrices(shape):
    zero = torch.zeros(shape, device=DEV)
    for eps in (1e-7, 1e-45, 1e-300, 5e-324):
        assert (fw.orthogonalize_ns(zero, eps=eps) == 0).all()
        assert (fw.orthogonalize_ns(zero, steps=0, eps=eps) == 0).all()
    for steps in (0, 5):  # 0 / 0
        assert torch.isnan(fw.orthogonalize_ns(zero, steps=steps, eps=0.0)).all()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_ns_of_infinities(shape):
    g = normal(*shape, seed=5)
    g[..., 1, 2] = float("inf")
    assert torch.isnan(fw.orthogonalize_ns(g)).all()
    # no step: G / inf, which is 0, and NaN for the infinity itself
    out = fw.orthogonalize_ns(g, steps=0)
    assert torch.isnan(out[..., 1, 2]).all() and int(torch.isnan(out).sum()) == out[..., 1, 2].numel()
    assert (out[~torch.isnan(out)] == 0).all()
    g[..., 1, 2] = float("nan")
    assert torch.isnan(fw.orthogonalize_ns(g, steps=0)).all()


@pytest.mark.parametrize("line", ["row", "column"])
@pytest.mark.parametrize("power", [-3, -5, -6, -7])
@pytest.mark.parametrize("shape", [(256, 1024), (60, 1500), (900, 500)], ids=str)
def test_ns_keeps_rows_and_columns_far_below_the_others(shape, power, line):
    g = _ns.with_small(shape, line, power)
    exact = plain.newton_schulz(g)
    got = fw.orthogonalize_ns(g.to(DEV)).cpu()
    pick = (lambda v: v[7]) if line == "row" else (lambda v: v[:, 7])
    # a bfloat16 rounding and 1.45 times it in all; below 10^-6, where binary16
    # ends (X's entries near 10^-7 / sqrt(rows * columns) times 2^14 are some
    # forty of its smallest steps), two in a hundred
    assert _ns.distance(pick(got), pick(exact)) <= (0.02 if power < -6 else 1.6 * 1.7e-3)


@pytest.mark.parametrize("coefficients", [(1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (0.01, 0.0, 0.0), (1.0, 0.0, 0.0),
                                          (0.0, 1.0, 0.0), (-2.0, 0.5, 0.25), (0.5, 3.0, 0.0), (3.0, 4.0, 30.0),
                                          (8.0, -20.0, 13.0)], ids=str)
@pytest.mark.parametrize("shape", [(100, 300), (40, 900)], ids=str)
def test_ns_of_other_polynomials(shape, coefficients):
    """Growing, shrinking and unlike ones: each has its own ranges.  Of two the
    bounds run away while these matrices' values stay small."""
    g = _ns.noise(shape)
    kw = dict(steps=2 if coefficients[0] == 0 else 3, coefficients=coefficients)
    exact, host = plain.newton_schulz(g, **kw), _ns.held(g, **kw)
    got = fw.orthogonalize_ns(g.to(DEV), **kw)
    # a polynomial that blows values up past 65504 is outside what the operator
    # holds, and says so
    if not torch.isfinite(host).all():
        assert not torch.isfinite(got).any()
        return
    assert torch.isfinite(got).all()
    assert _ns.distance(got, exact) <= _ns.SAME * _ns.distance(host.bfloat16(), exact) + 2.0 ** -10
    if coefficients == (1.0, 0.0, 0.0):
        assert _ns.distance(got, exact) <= 1.2 * _ns.own_rounding(exact)


@pytest.mark.parametrize("power, off", [(-5, 1.6 * 1.7e-3), (-6, 8e-3), (-7, 0.08)])
def test_ns_keeps_rows_of_a_large_matrix_as_documented(power, off):
    """4096 x 4096, whose entries are near 2^-12: one of a row 10^-7 of the others
    is 2^14 * 2^-12 * 10^-7 = 4e-7, seven of binary16's smallest steps, which round
    it by 0.29 of one on average (4%; 0.4% for 10^-6), and the steps after it,
    of entries that have grown, by less."""
    g = normal(4096, 4096, seed=6)
    g[7] *= 10.0 ** power
    x = g.double()
    x = x / (x.norm() + 1e-7)
    a, b, c = _ns.MUON
    for _ in range(5):
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    assert _ns.distance(fw.orthogonalize_ns(g)[7], x[7].cpu()) <= off
