"""The operators beside autograd: they take no part in it, and a backward pass
that would need their gradients raises instead of leaving them out."""
from __future__ import annotations

import pytest
import torch

import dense_fp16_gemm_04_amd as fw
from dense_fp16_gemm_04_amd import operators
from test_operators import gated_inputs, normal, w4_inputs


def test_a_result_without_gradients_raises_in_the_backward_pass():
    leaf = torch.ones(3, requires_grad=True)
    y = torch.full((3,), 2.0)
    assert operators._without_gradients(y, "none", torch.ones(3), None) is y
    with torch.no_grad():
        assert operators._without_gradients(y, "none", leaf, None) is y
    z = operators._without_gradients(y, "has no gradients", torch.ones(3), leaf, None)
    assert (z == 2).all() and z.requires_grad
    with pytest.raises(RuntimeError, match="has no gradients"):
        (z * 2 + leaf).sum().backward()


@pytest.mark.gpu
def test_calls_with_inputs_that_require_gradients():
    x, wg, wu = gated_inputs(20, 64, 48, torch.float16, seed=1)
    xs, q, s, z = w4_inputs(3, 40, 64, 32, "whole", torch.float16)
    g = normal(70, 90, seed=2)
    want = [fw.gated_nt(x, wg, wu), fw.orthogonalize_ns(g), fw.gemv_w4(xs, q, s, z)]
    h, saved = fw.gated_nt_train(x, wg, wu)
    dh = normal(20, 48, seed=3, t=torch.float16)
    grads = fw.gated_nt_backward(dh, x, wg, wu, saved)
    for v in (wg, g, s):
        v.requires_grad_()
    calls = [lambda **kw: fw.gated_nt(x, wg, wu, **kw), lambda **kw: fw.orthogonalize_ns(g, **kw),
             lambda **kw: fw.gemv_w4(xs, q, s, z, **kw)]
    for call, w, name in zip(calls, want, ("gated_nt_backward", "orthogonalize_ns", "gemv_w4")):
        y = call()
        assert torch.equal(y, w)
        with pytest.raises(RuntimeError, match=name):
            y.float().sum().backward()
        with torch.no_grad():
            y = call()
        assert torch.equal(y, w) and not y.requires_grad
        out = torch.zeros_like(w)
        assert call(out=out) is out and torch.equal(out, w) and not out.requires_grad
    # the training pair gives its gradients itself
    h2, saved = fw.gated_nt_train(x, wg, wu)
    assert torch.equal(h2, h) and not h2.requires_grad
    for a, b in zip(fw.gated_nt_backward(dh, x, wg, wu, saved), grads):
        assert torch.equal(a, b) and not a.requires_grad
