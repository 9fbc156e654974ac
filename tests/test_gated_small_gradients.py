"""The gated layer's gradients for dH of any size: as near the exact ones as
their roundings allow, from binary16's smallest values to its largest."""
from __future__ import annotations

import pytest
import torch

import _operators as plain
import dense_fp16_gemm_04_amd as fw
from test_operators import DEV, _built, framed, gated_inputs, normal  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(512, 136, 200), (70, 65, 33), (1000, 264, 513), (5, 64, 2000), (2048, 256, 72)]


def rms(v):
    return float(v.square().mean().sqrt())


def compare(dh, x, wg, wu, act):
    """Each gradient within twice what rounding it alone leaves, on average: the
    rounding of dG and dU adds as much again (sqrt 2 in all, of independent
    errors of one size), and what dG and dU lose below 2^-11 of dH's largest
    entry, at most 2^-25 of 2^-4 (a step there), is 2^-10 of a rounding of
    entries a thousandth of the largest."""
    _, saved = fw.gated_nt_train(x, wg, wu, activation=act)
    got = fw.gated_nt_backward(dh, x, wg, wu, saved)
    want, bounds = plain.gated_gradients(dh, x, wg, wu, act)
    for name, g, w, b in zip(("dx", "dw_gate", "dw_up"), got, want, bounds):
        rounded = w.to(dh.dtype)
        there = torch.isfinite(rounded) & (w.abs() < 60000 if dh.dtype == torch.float16 else True)
        assert there.double().mean() > 0.5
        own = (rounded.double() - w)[there]
        err = (g.double().cpu() - w)[there]
        assert rms(err) <= 2 * rms(own), (name, rms(err), rms(own), rms(w))
    return got


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("std", [1e-7, 1e-6, 1e-5, 1e-3, 1.0, 30.0, 1000.0])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients_of_any_size(shape, std, act, t):
    T, D, F = shape
    t = plain.TYPES[t]
    x, wg, wu = gated_inputs(T, D, F, t, seed=sum(shape))
    if std > 100:
        x = (x.float() * 0.25).to(t)  # (so that most of dW stays in range)
    dh = normal(T, F, seed=7, std=std, t=t)
    compare(dh, x, wg, wu, act)


@pytest.mark.parametrize("std", [1e-6, 1e-5])
def test_a_last_gradient_far_above_the_others(std):
    """One entry a hundred times the rest sets the power of two."""
    x, wg, wu = gated_inputs(512, 136, 200, torch.float16, seed=1)
    dh = normal(512, 200, seed=8, std=std, t=torch.float16)
    dh[511, 199] = 100 * std
    compare(dh, x, wg, wu, "silu")


def test_products_past_binary16s_range():
    """dH times P and Q is out of binary16's range, the gradients of x are not."""
    T, D, F = 40, 64, 96
    x, wg, wu = gated_inputs(T, D, F, torch.float16, seed=2)
    x = (x.float() * 8).half()
    wg, wu = (w.half() for w in (wg.float() * 0.5, wu.float() * 0.5))
    dh = normal(T, F, seed=9, t=torch.float16).sign() * 30000
    _, saved = fw.gated_nt_train(x, wg, wu)
    dx, _, _ = fw.gated_nt_backward(dh * 0.03125, x, wg, wu, saved)
    big = fw.gated_nt_backward(dh, x, wg, wu, saved)[0]
    there = dx.float().abs() < 1900
    assert there.any() and torch.equal(big[there].float(), dx[there].float() * 32)


def test_infinite_gradients_keep_to_their_rows():
    """They do not set the power of two for the others."""
    x, wg, wu = gated_inputs(70, 72, 90, torch.float16, seed=3)
    dh = normal(70, 90, seed=10, std=1e-5, t=torch.float16)
    _, saved = fw.gated_nt_train(x, wg, wu)
    clean = fw.gated_nt_backward(dh, x, wg, wu, saved)
    for v in (float("inf"), float("nan"), float("-inf")):
        bad = dh.clone()
        row = int(torch.randint(1, 69, (1,), generator=torch.Generator().manual_seed(5)))
        bad[row, 3] = v
        assert float(bad[row].abs().nan_to_num(0, 0, 0).max()) <= float(dh.abs().max())
        dx, dwg, dwu = fw.gated_nt_backward(bad, x, wg, wu, saved)
        keep = [r for r in range(70) if r != row]
        assert torch.equal(dx[keep], clean[0][keep]) and not torch.isfinite(dx[row]).any()
        cols = [c for c in range(90) if c != 3]
        assert torch.equal(dwg[cols], clean[1][cols]) and torch.equal(dwu[cols], clean[2][cols])
        assert not torch.isfinite(dwu[3]).any()


def test_zero_gradients_and_views():
    x, wg, wu = gated_inputs(37, 72, 51, torch.float16, seed=4)
    _, saved = fw.gated_nt_train(x, wg, wu)
    for g in fw.gated_nt_backward(torch.zeros(37, 51, dtype=torch.float16, device=DEV), x, wg, wu, saved):
        assert (g == 0).all()
    dh = normal(37, 51, seed=11, std=1e-6, t=torch.float16)
    want = fw.gated_nt_backward(dh, x, wg, wu, saved)
    for offset in (0, 1):  # (what surrounds a view is not looked at)
        got = fw.gated_nt_backward(framed(dh, offset=offset, fill=1000.0)[0], x, wg, wu, saved)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
