"""Dropout on an MI355X, through the public entry points, against the 64-bit
form of ``_training`` and its own statistics."""
from __future__ import annotations

import os

import numpy as np
import pytest
import torch

import _training as plain
import dense_fp16_gemm_04_amd as fw
from dense_fp16_gemm_04_amd import build, operators
from test_operators import frame_intact, framed, normal

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not all(os.path.exists(operators.library_path(n)) for n in build.STEP_OPERATORS):
        import __graft_entry__
        __graft_entry__.build()


SHAPES = [(1, 1), (1, 7), (7, 1), (1, 8), (1, 9), (3, 5), (5, 8), (9, 11), (2, 16), (17, 24), (33, 100), (64, 129), (1000, 31), (3, 4099),
          (40, 1024)]


@pytest.mark.parametrize("t", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_values_and_mask(shape, t):
    x, r = normal(*shape, seed=1, t=plain.TYPES[t]), normal(*shape, seed=2, t=plain.TYPES[t])
    x[x == 0] = 1
    for p, seed, offset in ((0.1, 12345, 0), (0.5, (1 << 64) - 1, (1 << 64) - 1), (0.75, 1 << 40, 3), (0.0, 7, 7), (1.0, 7, 7)):
        want, bound = plain.dropout(x, p, seed, offset)
        got = fw.dropout(x, p, seed, offset)
        plain.assert_within(got, want, bound)
        assert torch.equal(got.cpu() == 0, want == 0)
        assert torch.equal(fw.dropout_backward(x, p, seed, offset), got)
        want, bound = plain.dropout(x, p, seed, offset, r)
        plain.assert_within(fw.dropout(x, p, seed, offset, residual=r), want, bound)
    assert torch.equal(fw.dropout(x, 0.0, 5), x) and (fw.dropout(x, 1.0, 5) == 0).all()
    assert torch.equal(fw.dropout(x, 1.0, 5, residual=r), r)


def test_p_is_held_to_sixteen_bits():
    x = torch.ones(1, 4096, device=DEV)
    for p in (1e-5, 2.0 ** -17 * 0.99, 2.0 ** -17, 2.0 ** -16, 0.3, 1 - 2.0 ** -16, 1 - 2.0 ** -18):
        want, bound = plain.dropout(x, p, 99)
        plain.assert_within(fw.dropout(x, p, 99), want, bound)


@pytest.mark.parametrize("p", [0.02, 0.1, 0.5, 0.9])
def test_the_mask_is_random(p):
    """Shares, over all elements and over each place in a block, and pairs of
    neighbours, within six deviations; another seed or offset, another mask."""
    n = 1 << 22
    x = torch.ones(1, n, device=DEV)
    mask = (fw.dropout(x, p, 2024, 1)[0] != 0).double()
    q = 1 - round(p * 65536) / 65536

    def share(m, expect):
        assert abs(float(m.mean()) - expect) <= 6 * (expect * (1 - expect) / m.numel()) ** 0.5

    share(mask, q)
    for i in range(8):
        share(mask[i::8], q)
    for d in (1, 2, 8, 64, 2048):
        pairs = mask.reshape(-1, 2, d)
        share(pairs[:, 0] * pairs[:, 1], q * q)
    for seed, offset in ((2025, 1), (2024, 2), (2024, 1 + (1 << 32)), (2024 + (1 << 32), 1)):
        share(mask * (fw.dropout(x, p, seed, offset)[0] != 0), q * q)


@pytest.mark.parametrize("shape", [(40, 64), (9, 333), (6, 4099), (50, 3), (7, 8)], ids=str)
@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("t", ["fp16", "fp32"])
def test_views_draw_the_same_mask(shape, offset, t):
    x, r = normal(*shape, seed=3, t=plain.TYPES[t]), normal(*shape, seed=4, t=plain.TYPES[t])
    want = fw.dropout(x, 0.3, 11, 12, residual=r)
    vx, vr = framed(x, offset=offset)[0], framed(r, cols=3, offset=offset)[0]
    vy, big = framed(torch.zeros_like(x), cols=5, offset=offset)
    assert fw.dropout(vx, 0.3, 11, 12, residual=vr, out=vy) is vy
    assert torch.equal(vy, want) and frame_intact(vy, big)
    assert torch.equal(fw.dropout(vx, 0.3, 11, 12, residual=r), want)
    # in place, of x and of the residual, in views and not
    for same in (x.clone(), framed(x, offset=offset)[0]):
        assert torch.equal(fw.dropout(same, 0.3, 11, 12, residual=r, out=same), want)
    for same in (r.clone(), framed(r, offset=offset)[0]):
        assert torch.equal(fw.dropout(vx, 0.3, 11, 12, residual=same, out=same), want)
    assert torch.equal(fw.dropout(x, 0.3, 11, 12, residual=x), (fw.dropout(x, 0.3, 11, 12, residual=x.clone())))


def test_what_is_dropped_is_gone():
    """NaN and infinities among dropped elements leave no trace, among kept ones they stay."""
    x, r = normal(50, 77, seed=5, t=torch.bfloat16), normal(50, 77, seed=6, t=torch.bfloat16)
    keep = torch.from_numpy(plain.kept(np.arange(50 * 77), 0.5, 8, 9)).reshape(50, 77).to(DEV)
    want = fw.dropout(x, 0.5, 8, 9, residual=r)
    for v in (float("nan"), float("inf"), float("-inf")):
        bad = torch.where(keep, x, torch.full_like(x, v))
        assert torch.equal(fw.dropout(bad, 0.5, 8, 9, residual=r), want)
        y = fw.dropout(torch.full_like(x, v), 0.5, 8, 9)
        assert (y[~keep] == 0).all() and not torch.isfinite(y[keep]).any()


def test_numbers_from_the_gpu():
    x = normal(20, 100, seed=7)
    for seed, offset, more in ((5, 6, 0), (-3, 6, 10), (1 << 62, -1, 5)):
        state = torch.tensor([seed, offset], device=DEV)
        want = fw.dropout(x, 0.4, seed % (1 << 64), (offset + more) % (1 << 64))
        assert torch.equal(fw.dropout(x, 0.4, state, more), want)
        assert torch.equal(fw.dropout_backward(x, 0.4, state, more), want)


def test_a_captured_graph_draws_anew():
    x, r = normal(30, 1001, seed=8, t=torch.float16), normal(30, 1001, seed=9, t=torch.float16)
    state = torch.tensor([77, 0], device=DEV)
    fw.dropout(x, 0.2, state)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = fw.dropout(x, 0.2, state, 1, residual=r)
        dx = fw.dropout_backward(y, 0.2, state, 1)
    for k in range(4):
        state[1] = 10 * k
        g.replay()
        torch.cuda.synchronize()
        want = fw.dropout(x, 0.2, 77, 10 * k + 1, residual=r)
        assert torch.equal(y, want) and torch.equal(dx, fw.dropout(want, 0.2, 77, 10 * k + 1))


def test_past_32_bits():
    """Elements, and blocks times eight, past 2^32: dense, and in rows whose pitch is longer."""
    rows, cols = 4200, 1 << 20
    x = torch.ones(rows, cols, dtype=torch.float16, device=DEV)
    y = fw.dropout(x, 0.5, 1, 2)
    for r in (0, 4095, 4096, 4199):
        want = torch.from_numpy(plain.kept(r * cols + np.arange(cols), 0.5, 1, 2))
        assert torch.equal(y[r].cpu() != 0, want)
    del y
    odd = fw.dropout(x[:, :cols - 3], 0.5, 1, 2)
    for r in (0, 4096, 4199):
        want = torch.from_numpy(plain.kept(r * (cols - 3) + np.arange(cols - 3), 0.5, 1, 2))
        assert torch.equal(odd[r].cpu() != 0, want)


def test_empty():
    for shape in ((0, 8), (4, 0), (0, 0)):
        x = torch.zeros(shape, dtype=torch.float16, device=DEV)
        assert fw.dropout(x, 0.5, 1).shape == shape and fw.dropout(x, 0.5, 1, residual=x).shape == shape


def test_refusals_on_gpu_tensors():
    x = normal(4, 16, seed=1)
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(ValueError, match="p must"):
            fw.dropout(x, p, 1)
    for seed, offset in ((-1, 0), (1 << 64, 0), (0, -1), (0, 1 << 64)):
        with pytest.raises(ValueError, match="2\\^64"):
            fw.dropout(x, 0.1, seed, offset)
    for state in (torch.zeros(2, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV), torch.zeros(2, dtype=torch.int64)):
        with pytest.raises((TypeError, ValueError), match="seed"):
            fw.dropout(x, 0.1, state)
    with pytest.raises(ValueError):
        fw.dropout(x, 0.1, 1, residual=x[:3])
    with pytest.raises(TypeError):
        fw.dropout(x, 0.1, 1, residual=x.half())
    with pytest.raises(TypeError):
        fw.dropout(x.double(), 0.1, 1)
    big = torch.zeros(8, 16, device=DEV)
    with pytest.raises(fw.GemmError):
        fw.dropout(big[:4], 0.1, 1, out=big[1:5])
    with pytest.raises(fw.GemmError):
        fw.dropout(x, 0.1, 1, residual=big[:4], out=big[1:5])
    with pytest.raises(fw.GemmError):
        fw.dropout(big[:4, :8], 0.1, 1, out=big.view(-1)[:32].view(4, 8))
