"""The gated layer and the 4-bit product within bounds near their roundings, at
the lengths where K is split over waves and workgroups; and, on the host, that
these bounds reject what a fault would leave."""
from __future__ import annotations

import pytest
import torch

import _operators as plain
import _tight
import dense_fp16_gemm_04_amd as fw
import test_operators as listed
from _tight import RESULT, gradient_times, near

DEV = "cuda:0"
FEW = [(1, 4096, 24), (2, 2056, 4100), (5, 1000, 333), (8, 72, 8200), (16, 8192, 130), (17, 4096, 100), (32, 1032, 331),
       (31, 8192, 9), (13, 33, 5000)]
LONG = [(300, 296, 5001), (304, 301, 5000), (5003, 296, 136), (600, 1032, 2736), (513, 1024, 2056)]
GATED = listed.GATED_SHAPES + FEW + LONG
W4 = listed.W4_SHAPES + listed.W4_MANY + [(1, 300, 8192, 128), (16, 520, 8192, 64), (5, 200, 6016, 32), (256, 130, 4096, 128)]


def on_cpu(make, *args, **kw):
    """What the GPU tests make, on the CPU."""
    there, listed.DEV = listed.DEV, "cpu"
    try:
        return make(*args, **kw)
    finally:
        listed.DEV = there


def lacking(v, want, bound, t, times):
    """A result that lacks something is not near: entry by entry in one of a
    hundred places at least, or on average where there are enough."""
    return not near(v, want, bound, times, t)


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [s for s in GATED if max(s) <= 8200 and s[0] * s[1] * s[2] <= 10 ** 9], ids=str)
def test_gated_bounds_reject_faults(shape, t):
    T, D, F = shape
    t = plain.TYPES[t]
    x, wg, wu = on_cpu(listed.gated_inputs, T, D, F, t, seed=sum(shape))
    want, bound = _tight.gated(x, wg, wu, "silu")
    assert near(want.to(t), want, bound, RESULT, t)
    assert lacking(torch.zeros_like(want), want, bound, t, RESULT)
    step = min(64, (D + 1) // 2)  # a step of K, the last one
    if D > 1:
        assert lacking(_tight.gated(x[:, :-step], wg[:, :-step], wu[:, :-step], "silu")[0].to(t), want, bound, t, RESULT)
    dh = on_cpu(listed.normal, T, F, seed=99, std=0.5, t=t)
    want, bounds = _tight.gradients(dh, x, wg, wu, "silu")
    for w, b in zip(want, bounds):
        assert near(w.to(t), w, b, gradient_times(T, F), t)
        assert lacking(torch.zeros_like(w), w, b, t, gradient_times(T, F))
    if F > 1:
        step = min(64, (F + 1) // 2)
        part = _tight.gradients(dh[:, :-step], x, wg[:-step], wu[:-step], "silu")[0][0]
        assert lacking(part.to(t), want[0], bounds[0], t, gradient_times(T, F))
    if T > 1:
        step = min(64, (T + 1) // 2)
        for i in (1, 2):
            part = _tight.gradients(dh[:-step], x[:-step], wg, wu, "silu")[0][i]
            assert lacking(part.to(t), want[i], bounds[i], t, gradient_times(T, F))


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("zeros", [None, "whole", "any"])
@pytest.mark.parametrize("shape", W4, ids=str)
def test_w4_bounds_reject_faults(shape, zeros, t):
    M, N, K, group = shape
    t = plain.TYPES[t]
    x, q, s, z = on_cpu(listed.w4_inputs, min(M, 70), min(N, 520), K, group, zeros, t, seed=sum(shape))
    want, bound = _tight.product_w4(x, q, s, z)
    assert near(want.to(t), want, bound, RESULT, t)
    assert lacking(torch.zeros_like(want), want, bound, t, RESULT)
    if K > 32:  # a run of 32 k
        less = x.clone()
        less[:, -32:] = 0
        assert lacking(_tight.product_w4(less, q, s, z)[0].to(t), want, bound, t, RESULT)
    # scales of the next group, and a zero point left out
    if s.shape[1] > 1:
        assert lacking(_tight.product_w4(x, q, s.roll(1, 1), z)[0].to(t), want, bound, t, RESULT)
    if z is not None and not (z == 8).all():
        assert lacking(_tight.product_w4(x, q, s, None)[0].to(t), want, bound, t, RESULT)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("shape", GATED, ids=str)
def test_gated_is_near(shape, act, t):
    T, D, F = shape
    t = plain.TYPES[t]
    x, wg, wu = listed.gated_inputs(T, D, F, t, seed=sum(shape))
    h, saved = fw.gated_nt_train(x, wg, wu, activation=act)
    want, bound = _tight.gated(x, wg, wu, act)
    plain.assert_within(h, want, bound, "h")
    assert near(h, want, bound, RESULT, t), "h"
    dh = listed.normal(T, F, seed=99, std=0.5, t=t)
    got = fw.gated_nt_backward(dh, x, wg, wu, saved)
    want, bounds = _tight.gradients(dh, x, wg, wu, act)
    for name, g, w, b in zip(("dx", "dw_gate", "dw_up"), got, want, bounds):
        plain.assert_within(g, w, b, name)
        assert near(g, w, b, gradient_times(T, F), t), name


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("zeros", [None, "whole", "any"])
@pytest.mark.parametrize("shape", W4, ids=str)
def test_w4_is_near(shape, zeros, t):
    M, N, K, group = shape
    t = plain.TYPES[t]
    x, q, s, z = listed.w4_inputs(M, N, K, group, zeros, t, seed=sum(shape))
    want, bound = _tight.product_w4(x, q, s, z)
    for offset in (0, 1):
        got = fw.gemv_w4(listed.framed(x, offset=offset)[0], q, s, z)
        plain.assert_within(got, want, bound)
        assert near(got, want, bound, RESULT, t)
