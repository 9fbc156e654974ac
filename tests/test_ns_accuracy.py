"""Newton-Schulz against the exact iteration: the error that the documented
roundings have on the host, and no more, for noise and for singular values that
fall off."""
from __future__ import annotations

import pytest
import torch

import _ns
import _operators as plain
import dense_fp16_gemm_04_amd as fw

DEV = "cuda:0"

# tiles of every size, split sums, one launch a step; wide and tall
SHAPES = [(54, 1286), (40, 4000), (64, 64), (33, 8192), (8000, 24), (65, 63), (256, 256), (320, 320), (130, 700),
          (512, 520), (1536, 1030), (300, 9000)]


@pytest.mark.parametrize("shape", SHAPES[:10], ids=str)
def test_host_form_and_what_the_bounds_reject(shape):
    g = _ns.noise(shape)
    exact, host = plain.newton_schulz(g), _ns.held(g)
    limit = _ns.SAME * _ns.distance(host.bfloat16(), exact)
    assert limit <= 1.45 * _ns.own_rounding(exact)
    assert _ns.distance(_ns.held(g, corrected=False).bfloat16(), exact) > limit
    bound = _ns.entry_bound(exact, host)
    got = host.bfloat16().double()
    assert ((got - exact).abs() <= bound).all()
    # sixteen entries lost at the end of the last row, or anywhere
    assert ((exact.abs() > bound)[-1, -16:]).any()
    assert float((exact.abs() > bound).double().mean()) > 0.9


@pytest.mark.parametrize("tens, ratio", [(1, 1.3), (2, 3.0), (4, 7.0), (6, 9.0)])
def test_host_form_of_decaying_singular_values(tens, ratio):
    g = _ns.decaying((256, 1024), tens)
    exact = plain.newton_schulz(g)
    assert ratio / 2 < _ns.distance(_ns.held(g).bfloat16(), exact) / _ns.own_rounding(exact) < ratio


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_ns_is_as_near_the_exact_iteration_as_documented(shape, t):
    g = _ns.noise(shape, plain.TYPES[t])
    exact, host = plain.newton_schulz(g), _ns.held(g)
    got = fw.orthogonalize_ns(g.to(DEV))
    plain.assert_within(got, exact, _ns.entry_bound(exact, host))
    assert _ns.distance(got, exact) <= _ns.SAME * _ns.distance(host.bfloat16(), exact)
    assert _ns.distance(got, exact) <= 1.45 * _ns.own_rounding(exact)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(64, 16500), (33, 100001), (150000, 5), (1, 70000), (3, 20, 20000)], ids=str)
def test_ns_of_few_long_rows(shape):
    """Sixty-four rows or fewer, of any length."""
    g = _ns.noise(shape)
    got = fw.orthogonalize_ns(g.to(DEV)).cpu()
    for a, b in zip(g if g.dim() == 3 else [g], got if g.dim() == 3 else [got]):
        exact, host = plain.newton_schulz(a), _ns.held(a)
        plain.assert_within(b, exact, _ns.entry_bound(exact, host))
        assert _ns.distance(b, exact) <= _ns.SAME * _ns.distance(host.bfloat16(), exact)
    assert torch.equal(got, fw.orthogonalize_ns(g.to(DEV)).cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1100, 2900), (2, 520, 2000), (9, 1024, 1280)], ids=str)
def test_ns_large_is_as_near_the_exact_iteration_as_documented(shape):
    """Two steps (the host's 64-bit products take long)."""
    g = _ns.noise(shape, torch.bfloat16)
    got = fw.orthogonalize_ns(g.to(DEV), steps=2).cpu()
    for a, b in [(g, got)] if g.dim() == 2 else [(g[0], got[0]), (g[-1], got[-1])]:
        exact, host = plain.newton_schulz(a, steps=2), _ns.held(a, steps=2)
        plain.assert_within(b, exact, _ns.entry_bound(exact, host))
        assert _ns.distance(b, exact) <= _ns.SAME * _ns.distance(host.bfloat16(), exact)


@pytest.mark.gpu
@pytest.mark.parametrize("tens", [1, 2, 4, 6])
@pytest.mark.parametrize("shape", [(256, 1024), (60, 1500), (900, 500)], ids=str)
def test_ns_of_decaying_singular_values(shape, tens):
    g = _ns.decaying(shape, tens)
    exact, host = plain.newton_schulz(g), _ns.held(g)
    got = fw.orthogonalize_ns(g.to(DEV))
    assert _ns.distance(got, exact) <= _ns.SAME * _ns.distance(host.bfloat16(), exact)
    plain.assert_within(got, exact, _ns.entry_bound(exact, host))
