"""Newton-Schulz at the ends of G's range: norms whose inverse 32 bits cannot
hold, zero matrices, infinities."""
from __future__ import annotations

import pytest
import torch

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
