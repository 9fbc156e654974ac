"""The operators of a training step together on an MI355X: a feed-forward block
between its norm, dropout and residual, under the loss over a vocabulary; on
streams, in graphs, repeated, and beside autograd."""
from __future__ import annotations

import os

import pytest
import torch
from torch.autograd import forward_ad

import _training as plain
import dense_fp16_gemm_04_amd as fw
from dense_fp16_gemm_04_amd import build, operators, training
from test_operators import normal

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
P = 0.1


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not all(os.path.exists(operators.library_path(n)) for n in build.OPERATORS + build.STEP_OPERATORS):
        import __graft_entry__
        __graft_entry__.build()


def inputs(T, D, F, V, t, seed):
    target = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(seed)).to(DEV)
    target[::7] = -100
    return [normal(T, D, seed=seed + 1, t=t), normal(D, seed=seed + 2, std=0.1, t=torch.float32) + 1, normal(D, seed=seed + 3, std=0.1),
            normal(F, D, seed=seed + 4, std=D ** -0.5, t=t), normal(F, D, seed=seed + 5, std=D ** -0.5, t=t),
            normal(D, F, seed=seed + 6, std=F ** -0.5, t=t), normal(V, D, seed=seed + 7, std=D ** -0.5, t=t), target,
            torch.tensor([seed, 5], device=DEV)]


def step(x, nw, nb, wg, wu, wd, wo, target, state, scale=256.0):
    """x + dropout(down(gated(norm(x)))), norm, loss; the gradients of scale times its sum of all
    but the down projection's weight: [loss, dx, dnw, dnb, dwg, dwu, dwo]."""
    n, n_saved = fw.layer_norm_train(x, nw, nb)
    h, h_saved = fw.gated_nt_train(n, wg, wu)
    f = fw.gemm_nt_f16(h, wd)
    r = fw.dropout(f, P, state, 1, residual=x)
    m, m_saved = fw.layer_norm_train(r, nw, None)
    loss, l_saved = fw.linear_cross_entropy_train(m, wo, target)
    g = torch.full((1,), scale, device=DEV).expand(x.shape[0])
    dm, dwo = fw.linear_cross_entropy_backward(g, m, wo, target, l_saved)
    dr, dnw, _ = fw.layer_norm_backward(dm, r, nw, None, m_saved)
    df = fw.dropout_backward(dr, P, state, 1)
    dh = fw.gemm_nt_f16(df, wd.t().contiguous())
    dn, dwg, dwu = fw.gated_nt_backward(dh, n, wg, wu, h_saved)
    dx, dnw2, dnb = fw.layer_norm_backward(dn, x, nw, nb, n_saved)
    return [loss, dx.add_(dr), dnw.add_(dnw2), dnb, dwg, dwu, dwo]


def step64(x, nw, nb, wg, wu, wd, wo, target, state, scale=256.0):
    """The same in 64 bits, by autograd."""
    leaves = [v.double().requires_grad_() for v in (x, nw, nb, wg, wu, wo)]
    x64, nw64, nb64, wg64, wu64, wo64 = leaves

    def norm(v, w, b):
        c = v - v.mean(1, keepdim=True)
        return c / (c.square().mean(1, keepdim=True) + 1e-5).sqrt() * w + b

    n = norm(x64, nw64, nb64)
    g = n @ wg64.T
    f = (g * torch.sigmoid(g) * (n @ wu64.T)) @ wd.double().T
    seed, offset = (int(v) for v in state.cpu())
    keep = torch.from_numpy(plain.kept(range(x.numel()), P, seed, offset + 1)).reshape(x.shape).to(DEV)
    q = 1 - round(P * 65536) / 65536
    r = x64 + torch.where(keep, f / q, torch.zeros_like(f))
    l = norm(r, nw64, 0.0) @ wo64.T
    valid = target != -100
    loss = torch.where(valid, torch.logsumexp(l, 1) - l.gather(1, target.clamp(min=0)[:, None])[:, 0], torch.zeros_like(l[:, 0]))
    grads = torch.autograd.grad(scale * loss.sum(), leaves)
    return [loss.detach(), *grads]


@pytest.mark.parametrize("shape", [(96, 256, 320, 500), (200, 136, 264, 1001)], ids=str)
def test_a_step_against_64_bits(shape):
    """Every stage rounds to binary16 at half a step of 2^-11; a gradient passes
    through about a dozen roundings of its factors, which mostly differ in
    sign: within 8 half steps of the whole (root of squares), the loss, behind
    five, within 5 of its size."""
    args = inputs(*shape, torch.float16, seed=50)
    got, want = step(*args), step64(*args)
    half = 2.0 ** -11
    for name, g, w, most in zip(("loss", "dx", "dnw", "dnb", "dwg", "dwu", "dwo"), got, want, (5, 8, 8, 8, 8, 8, 8)):
        off = float((g.double() - w).norm() / w.norm())
        assert off <= most * half, (name, off / half)


def test_steps_repeat_bit_for_bit():
    args = inputs(96, 256, 320, 500, torch.float16, seed=60)
    first = step(*args)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, step(*args)))


def test_streams_side_by_side():
    sets = [inputs(64 + 32 * i, 256, 320, 500 + i, torch.float16, seed=70 + i) for i in range(3)]
    want = [step(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None] * len(sets)
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = step(*sets[i])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_captured_graphs_replay():
    """Two graphs of a whole step, replayed in turn on changing inputs with
    eager steps between, against eager results."""
    shapes = [(96, 256, 320, 500), (33, 136, 264, 1001)]
    sets = [inputs(*s, torch.float16, seed=80 + i) for i, s in enumerate(shapes)]
    graphs, outs = [], []
    for args in sets:
        step(*args)  # libraries loaded, allocator warm
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*args))
        graphs.append(g)
    for k in range(4):
        for s, args, g, out in zip(shapes, sets, graphs, outs):
            for a, v in zip(args, inputs(*s, torch.float16, seed=100 + k)):
                a.copy_(v)
            g.replay()
            torch.cuda.synchronize()
            kept = [o.clone() for o in out]
            assert all(torch.equal(a, b) for a, b in zip(kept, step(*args)))


def many(x, w, b, dy, xl, wl, target, g):
    """The kernels of larger sizes: wide and narrow norms, several pieces and parts."""
    y, saved = fw.layer_norm_train(x, w, b)
    loss, l_saved = fw.linear_cross_entropy_train(xl, wl, target)
    return [y, *fw.layer_norm_backward(dy, x, w, b, saved), fw.dropout(x, 0.5, 3, 4, residual=dy), loss,
            *fw.linear_cross_entropy_backward(g, xl, wl, target, l_saved)]


def many_inputs(rows, cols, T, D, V, seed):
    target = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(seed)).to(DEV)
    t = torch.bfloat16
    return [normal(rows, cols, seed=seed, t=t), normal(cols, seed=seed + 1, t=t), normal(cols, seed=seed + 2, t=t),
            normal(rows, cols, seed=seed + 3, t=t), normal(T, D, seed=seed + 4, t=t), normal(V, D, seed=seed + 5, std=D ** -0.5, t=t), target,
            normal(T, seed=seed + 6)]


def test_large_calls_on_streams_and_in_graphs():
    shapes = [(300, 40000, 4101, 200, 4093), (9000, 24, 300, 8200, 1001), (500, 2731, 1, 64, 9000)]
    sets = [many_inputs(*s, seed=120 + i) for i, s in enumerate(shapes)]
    want = [many(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None] * len(sets)
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = many(*sets[i])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))
    graphs, outs = [], []
    for args in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(many(*args))
        graphs.append(g)
    for k in range(3):
        for s, args, g, out in zip(shapes, sets, graphs, outs):
            for a, v in zip(args, many_inputs(*s, seed=140 + k)):
                a.copy_(v)
            g.replay()
            torch.cuda.synchronize()
            kept = [o.clone() for o in out]
            assert all(torch.equal(a, b) for a, b in zip(kept, many(*args)))


@pytest.mark.parametrize("shape", [(300, 40000, 4101, 200, 4093), (9000, 24, 300, 8200, 1001), (500, 2731, 1, 64, 9000), (3, 8, 17, 4096, 20001),
                                   (3, 8, 200, 333, 30001), (3, 8, 4101, 1080, 4093), (3, 8, 9000, 136, 33001), (3, 8, 0, 16, 300),
                                   (0, 24, 40, 776, 2 ** 20 + 5003)], ids=str)
def test_nothing_is_written_past_a_workspace(shape, monkeypatch):
    args = many_inputs(*shape, seed=190)
    want = many(*args)
    given = []

    def framed(like, nbytes):
        given.append(torch.full((max(nbytes, 0) + 8192,), 0x5A, dtype=torch.uint8, device=like.device))
        return given[-1], given[-1].data_ptr() + 4096 if nbytes > 0 else None

    monkeypatch.setattr(training, "_workspace", framed)
    got = many(*args)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert len(given) == 3
    for w in given:
        assert (w[:4096] == 0x5A).all() and (w[-4096:] == 0x5A).all()


def test_on_another_current_device(monkeypatch):
    """The operand's device is entered when another one is current (simulated on one GPU)."""
    args = many_inputs(20, 64, 30, 64, 100, seed=160)
    want = many(*args)
    entered = []

    class Enter:
        def __init__(self, index):
            entered.append(index)

        def __enter__(self):
            return self

        def __exit__(self, *exc):
            return False

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", Enter)
    got = many(*args)
    monkeypatch.undo()
    assert entered == [0] * 5
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_inputs_that_require_gradients():
    x, w, b, dy, xl, wl, target, g = many_inputs(20, 64, 30, 64, 100, seed=170)
    want = many(x, w, b, dy, xl, wl, target, g)
    for v in (w, dy, wl):
        v.requires_grad_()
    calls = [(lambda **kw: fw.layer_norm(x, w, b, **kw), "layer_norm_backward"),
             (lambda **kw: fw.dropout(x, 0.5, 3, 4, residual=dy, **kw), "dropout_backward"),
             (lambda **kw: fw.linear_cross_entropy(xl, wl, target, **kw), "linear_cross_entropy_backward")]
    for (call, name), ref in zip(calls, (want[0], want[4], want[5])):
        y = call()
        assert torch.equal(y, ref)
        with pytest.raises(RuntimeError, match=name):
            y.float().sum().backward()
        with torch.no_grad():
            y = call()
        assert torch.equal(y, ref) and not y.requires_grad
        out = torch.zeros_like(ref)
        assert call(out=out) is out and torch.equal(out, ref) and not out.requires_grad
    # the training forms give their gradients themselves
    got = many(x, w, b, dy.detach(), xl, wl, target, g)
    assert all(torch.equal(a, c) and not a.requires_grad for a, c in zip(got, want))


def test_derivatives_that_a_call_does_not_have():
    """Tangents are refused; a second derivative raises when it is asked for."""
    x, w, b, dy, xl, wl, target, g = many_inputs(20, 64, 30, 64, 100, seed=180)
    want = many(x, w, b, dy, xl, wl, target, g)
    y, saved = fw.layer_norm_train(x, w, b)
    _, l_saved = fw.linear_cross_entropy_train(xl, wl, target)
    with forward_ad.dual_level():
        assert all(torch.equal(a, c) for a, c in zip(want, many(x, w, b, dy, xl, wl, target, g)))
        wd, xd, dd, gd = (forward_ad.make_dual(v, torch.ones_like(v)) for v in (w, xl, dy, g))
        for call in (lambda: fw.layer_norm(x, wd, b), lambda: fw.layer_norm_train(x, w, wd), lambda: fw.dropout(x, 0.5, 3, residual=dd),
                     lambda: fw.layer_norm_backward(dd, x, w, b, saved), lambda: fw.dropout_backward(dd, 0.5, 3),
                     lambda: fw.layer_norm(x, w, b, out=dd),
                     lambda: fw.linear_cross_entropy(xd, wl, target), lambda: fw.linear_cross_entropy_train(xl, wl, target, out=gd),
                     lambda: fw.linear_cross_entropy_backward(gd, xl, wl, target, l_saved)):
            with pytest.raises(RuntimeError, match="tangent"):
                call()
        assert all(torch.equal(a, c) for a, c in zip(want, many(x, w, b, dy, xl, wl, target, g)))
    plain_grads = [*fw.layer_norm_backward(dy, x, w, b, saved), fw.dropout_backward(dy, 0.5, 3),
                   *fw.linear_cross_entropy_backward(g, xl, wl, target, l_saved)]
    for v in (dy, g):
        v.requires_grad_()
    grads = [*fw.layer_norm_backward(dy, x, w, b, saved), fw.dropout_backward(dy, 0.5, 3),
             *fw.linear_cross_entropy_backward(g, xl, wl, target, l_saved)]
    for a, c in zip(grads, plain_grads):
        assert torch.equal(a, c)
        with pytest.raises(RuntimeError, match="_backward has no gradients"):
            a.float().sum().backward()
    out = [torch.zeros_like(c) for c in plain_grads]
    fw.layer_norm_backward(dy, x, w, b, saved, out=out[:3])
    fw.dropout_backward(dy, 0.5, 3, out=out[3])
    fw.linear_cross_entropy_backward(g, xl, wl, target, l_saved, out=out[4:])
    with torch.no_grad():
        grads = [*fw.layer_norm_backward(dy, x, w, b, saved), fw.dropout_backward(dy, 0.5, 3),
                 *fw.linear_cross_entropy_backward(g, xl, wl, target, l_saved)]
    assert all(torch.equal(a, c) and not a.requires_grad for a, c in zip(grads + out, 2 * plain_grads))
