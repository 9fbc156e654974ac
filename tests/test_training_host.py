"""The operators around a training step's products without a GPU: their
libraries export what the headers declare and refuse bad arguments before
enqueuing anything; the plain forms against published values and differences."""
from __future__ import annotations

import json
import os
import re

import pytest
import torch
from torch.autograd import forward_ad

import _training as plain
import dense_fp16_gemm_04_amd as fw
from dense_fp16_gemm_04_amd import build, operators, training

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID = 1  # hipErrorInvalidValue
# addresses that are never touched: 64 MiB apart, 16-byte aligned
A, B, C, D, E, F, G, H, W = (0x10000000 + i * 0x4000000 for i in range(9))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not all(os.path.exists(operators.library_path(n)) for n in build.STEP_OPERATORS):
        import __graft_entry__
        __graft_entry__.build()


@pytest.mark.parametrize("name", build.STEP_OPERATORS)
def test_declared_symbols_and_version(name):
    text = open(os.path.join(ROOT, "include", name + ".h")).read()
    declared = sorted(set(re.findall(r"\b(%s\w*)\s*\(" % name, re.sub(r"/\*.*?\*/", "", text, flags=re.S))))
    assert sorted(operators.SIGNATURES[name]) == declared
    version = re.search(r"#define\s+%s_VERSION\s+(\d+)" % name.upper(), text)
    assert getattr(operators.load(name), name + "_version")() == int(version.group(1))


@pytest.mark.parametrize("name", build.STEP_OPERATORS)
def test_no_kernel_spills(name):
    kernels = json.load(open(build.operator_paths(name)[2]))["kernels"]
    assert kernels and build.spilling(kernels) == []


@pytest.mark.parametrize("name", build.STEP_OPERATORS)
def test_wide_buffer_stores_take_no_scalar_offset(name, tmp_path):
    """(Why: tests/test_operators_host.py, the test of this name.)"""
    import _isa
    asm = _isa.disassemble(operators.library_path(name), tmp_path)
    stores = [l.split("//")[0].strip() for l in asm.splitlines() if re.search(r"\bbuffer_store_dwordx[34]\b", l)]
    assert [l for l in stores if not re.search(r", 0 (offen|idxen)|, off, s\[[0-9:]+\], 0", l)] == []


# ----------------------------------------------------------- layer_norm --

def norm_args(**kw):
    a = dict(X=A, weight=B, bias=C, Y=D, saved=E, rows=4, cols=16, ldx=16, ldy=16, type=0, param=0, eps=1e-5, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(rows=1 << 31), dict(cols=(1 << 24) + 1, ldx=1 << 25, ldy=1 << 25), dict(ldx=15), dict(ldy=15),
    dict(ldx=1 << 31), dict(ldy=1 << 31), dict(rows=(1 << 31) - 1, ldx=(1 << 31) - 1), dict(type=3), dict(type=-1), dict(param=1),
    dict(type=1, param=0), dict(type=2, param=0), dict(eps=-1e-9), dict(eps=float("nan")), dict(X=None), dict(Y=None), dict(X=A + 1),
    dict(Y=D + 1), dict(weight=B + 1), dict(weight=B + 2, param=2), dict(bias=C + 1), dict(saved=E + 4), dict(Y=A), dict(Y=A + 64),
    dict(Y=B), dict(Y=C), dict(saved=A), dict(saved=B), dict(saved=D), dict(X=A + 2, type=2, param=2),
])
def test_layer_norm_refuses(kw):
    assert operators.load("layer_norm").layer_norm(*norm_args(**kw)) == INVALID


def norm_back_args(**kw):
    a = dict(dY=A, X=B, weight=C, saved=D, dX=E, dweight=F, dbias=G, rows=4, cols=16, lddy=16, ldx=16, lddx=16, type=0, param=0, ws=W,
             ws_bytes=1 << 25, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(lddy=15), dict(ldx=15), dict(lddx=15), dict(type=3), dict(param=1), dict(dY=None), dict(X=None),
    dict(saved=None), dict(saved=D + 4), dict(dX=None), dict(dX=E + 1), dict(weight=C + 1), dict(dweight=F + 1), dict(dbias=G + 1),
    dict(ws=None), dict(ws_bytes=64), dict(ws=W + 8), dict(dX=A), dict(dX=B), dict(dX=D), dict(dweight=C), dict(dbias=F), dict(dweight=E),
    dict(ws=A), dict(ws=E), dict(cols=1 << 25, lddy=1 << 25, ldx=1 << 25, lddx=1 << 25),
])
def test_layer_norm_backward_refuses(kw):
    assert operators.load("layer_norm").layer_norm_backward(*norm_back_args(**kw)) == INVALID


def test_layer_norm_empty_and_workspace():
    lib = operators.load("layer_norm")
    assert lib.layer_norm(*norm_args(rows=0, X=None, Y=None)) == 0
    assert lib.layer_norm(*norm_args(cols=0, X=None, Y=None)) == 0
    assert lib.layer_norm_backward(*norm_back_args(cols=0, dY=None, X=None, dX=None)) == 0
    assert lib.layer_norm_backward_workspace(-1, 4) == -1 and lib.layer_norm_backward_workspace(4, (1 << 24) + 1) == -1
    assert lib.layer_norm_backward_workspace(4, 16) > 0


@pytest.mark.parametrize("cols", [20000, 1 << 19, (1 << 19) + 1, 1 << 22, 1 << 24])
def test_layer_norm_backward_workspace_of_wide_rows(cols):
    """Sums of columns of 256 MB at most (64 shares of 2^24 columns would be 8.6 GB beside rows of 2), two means a row."""
    assert 0 < operators.load("layer_norm").layer_norm_backward_workspace(64, cols) <= (1 << 28) + (1 << 14)


# -------------------------------------------------------------- dropout --

def dropout_args(**kw):
    a = dict(X=A, residual=B, Y=C, rows=4, cols=16, ldx=16, ldr=16, ldy=16, type=0, p=0.1, seed=1, offset=2, state=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(rows=1 << 31), dict(cols=1 << 31, ldx=1 << 31, ldr=1 << 31, ldy=1 << 31), dict(ldx=15), dict(ldr=15),
    dict(ldy=15), dict(ldx=1 << 31), dict(type=3), dict(type=-1), dict(p=-0.01), dict(p=1.01), dict(p=float("nan")), dict(X=None),
    dict(Y=None), dict(X=A + 1), dict(residual=B + 1), dict(Y=C + 1), dict(X=A + 2, type=2), dict(state=D + 4), dict(Y=A + 16),
    dict(Y=B + 16), dict(Y=A, ldx=17), dict(Y=B, ldr=17), dict(state=C), dict(Y=A, residual=A + 32),
])
def test_dropout_refuses(kw):
    assert operators.load("dropout").dropout(*dropout_args(**kw)) == INVALID


def test_dropout_empty_is_a_no_op():
    lib = operators.load("dropout")
    assert lib.dropout(*dropout_args(rows=0, X=None, Y=None)) == 0
    assert lib.dropout(*dropout_args(cols=0, X=None, Y=None)) == 0


def test_philox_gives_the_published_words():
    """The generator's known answers (counter, key, words), as its authors publish them."""
    ones = 0xFFFFFFFF
    known = [((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
             ((ones,) * 4, (ones,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
             ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]
    for counter, key, words in known:
        assert tuple(plain.philox([counter], key)[0]) == words


def test_the_plain_mask_follows_the_generator():
    p, seed, offset = 0.3, 0x123456789ABCDEF0, 0xFEDCBA9876543210
    at = list(range(40)) + [(1 << 35) + i for i in range(24)]
    want = []
    for e in at:
        b = e // 8
        words = plain.philox([(b & 0xFFFFFFFF, b >> 32, offset & 0xFFFFFFFF, offset >> 32)], (seed & 0xFFFFFFFF, seed >> 32))[0]
        want.append((words[e % 8 // 2] >> (16 * (e % 2)) & 0xFFFF) >= round(p * 65536))
    assert plain.kept(at, p, seed, offset).tolist() == want


# ------------------------------------------------------------- bindings --

def test_bindings_refuse_host_tensors_and_wrong_types():
    x = torch.zeros(4, 16)
    for call in (lambda: fw.layer_norm(x), lambda: fw.layer_norm_train(x), lambda: fw.dropout(x, 0.1, 1),
                 lambda: fw.layer_norm_backward(x, x, None, None, torch.zeros(4, 2)), lambda: fw.dropout_backward(x, 0.1, 1)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: fw.layer_norm(x.double()), lambda: fw.layer_norm([1.0]), lambda: fw.dropout(x.long(), 0.1, 1)):
        with pytest.raises(TypeError):
            call()


def test_entry_points_are_kept_by_library(monkeypatch):
    """Two libraries that export one name: each call reaches its own."""
    class Library:
        def __init__(self, code):
            self.entry = lambda *args: code

    libraries = {"first": Library(0), "second": Library(7)}
    monkeypatch.setattr(operators, "load", libraries.__getitem__)
    monkeypatch.setattr(operators, "_stream", lambda device: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for _ in range(2):
        operators._call("first", "entry", 0)
        with pytest.raises(fw.GemmError):
            operators._call("second", "entry", 0)


def test_tangents_are_refused():
    """A dual tensor of forward-mode differentiation, whose tangent a call would lose."""
    x, v, w = torch.zeros(4, 16), torch.ones(16), torch.zeros(8, 16)
    target, saved = torch.zeros(4, dtype=torch.int64), torch.zeros(4, 3)
    with forward_ad.dual_level():
        dual = [forward_ad.make_dual(t, torch.ones_like(t)) for t in (x, v, x.half())]
        for call in (lambda: fw.layer_norm(dual[0]), lambda: fw.layer_norm_train(dual[0], v, v), lambda: fw.dropout(dual[0], 0.1, 1),
                     lambda: fw.layer_norm_backward(x, dual[0], None, None, saved[:, :2]), lambda: fw.dropout_backward(dual[0], 0.1, 1),
                     lambda: fw.linear_cross_entropy(dual[2], w.half(), target), lambda: fw.linear_cross_entropy_train(dual[2], w.half(), target),
                     lambda: fw.linear_cross_entropy_backward(saved[:, 0], dual[2], w.half(), target, saved),
                     lambda: training._vector("weight", dual[1], (torch.float32,), -1, 16),
                     lambda: training._strided("dloss", dual[1], torch.float32, -1, 16),
                     lambda: fw.gated_nt(dual[2], w.half(), w.half()), lambda: fw.orthogonalize_ns(dual[0])):
            with pytest.raises(RuntimeError, match="tangent"):
                call()
        # others are looked at as ever
        training._vector("weight", v, (torch.float32,), -1, 16)
        with pytest.raises(ValueError, match="GPU"):
            fw.layer_norm(x)
        with pytest.raises(TypeError):
            fw.layer_norm([1.0])


# ------------------------------------------------- the plain forms here --

def test_plain_norm_gradients_match_differences():
    gen = torch.Generator().manual_seed(7)
    x, w, dy = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((5, 9), (9,), (5, 9)))
    grads, _ = plain.norm_gradients(dy, x, w)

    def loss(x, w, b):
        c = x - x.mean(1, keepdim=True)
        return ((c / (c.square().mean(1, keepdim=True) + 1e-5).sqrt() * w + b) * dy).sum()

    leaves = [x, w, torch.zeros(9, dtype=torch.float64)]
    for i in range(3):
        v = torch.randn(leaves[i].shape, generator=gen, dtype=torch.float64)
        ends = [loss(*(u + s * 1e-5 * v if k == i else u for k, u in enumerate(leaves))) for s in (1, -1)]
        slope = float(ends[0] - ends[1]) / 2e-5
        assert abs(slope - float((grads[i] * v).sum())) <= 1e-7 * max(1.0, abs(slope))


@pytest.mark.parametrize("cols", [7, 300, 5000, 70000])
@pytest.mark.parametrize("t", ["fp16", "bf16", "fp32"])
def test_norm_bounds_reject_what_is_wrong(cols, t):
    """Zeros, a missing element in the mean, a variance of n - 1, and a lost mean(g h)."""
    t = plain.TYPES[t]
    gen = torch.Generator().manual_seed(cols)
    x, dy = ((torch.randn(6, cols, generator=gen) * 2 + 0.5).to(t) for _ in range(2))
    y, bound = plain.norm(x, None, None)
    (dx, dw, db), bounds = plain.norm_gradients(dy, x, None)

    def outside(got, want, bound):
        return bool(((got - want).abs() > bound).any())

    for want, b in zip((y, dx, dw, db), (bound, *bounds)):
        assert outside(torch.zeros_like(want), want, b)
    d = x.double()
    # (what changes y by less than its rounding cannot be seen)
    fine = torch.finfo(t).eps if t != torch.float32 else 32 * torch.finfo(t).eps
    if 1 / cols > fine:
        c = d - d[:, 1:].sum(1, keepdim=True) / cols
        assert outside(c / (c.square().mean(1, keepdim=True) + 1e-5).sqrt(), y, bound)
    if 1 / (2 * cols) > fine:
        assert outside(y * ((cols - 1) / cols) ** 0.5, y, bound)
    g = dy.double()
    h = y
    r = 1 / (d.var(1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    lost = r * (g - g.mean(1, keepdim=True))
    if cols <= 300 or t == torch.float32 and cols <= 5000:
        assert outside(lost, dx, bounds[0])
    assert outside(dw - g[0] * h[0], dw, bounds[1]) and outside(db - g[0], db, bounds[2])


# ------------------------------------------------- linear_cross_entropy --

def loss_args(**kw):
    a = dict(X=A, W=B, target=C, loss=D, saved=E, T=4, D=16, V=8, ldx=16, ldw=16, stride=1, type=0, ignore=-100, ws=W, ws_bytes=1 << 25,
             stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(D=-1), dict(V=-1), dict(V=0), dict(T=(1 << 27) + 1), dict(V=1 << 31), dict(D=1 << 21, ldx=1 << 21, ldw=1 << 21), dict(ldx=15),
    dict(ldw=15), dict(ldx=1 << 21), dict(stride=-1), dict(stride=(1 << 31) + 1), dict(type=2), dict(type=-1), dict(X=None), dict(W=None),
    dict(target=None), dict(loss=None), dict(X=A + 1), dict(W=B + 1), dict(target=C + 4), dict(loss=D + 2), dict(saved=E + 2),
    dict(ws=None), dict(ws_bytes=64), dict(ws=W + 8), dict(loss=A), dict(loss=B), dict(loss=C), dict(saved=A), dict(saved=D), dict(ws=A),
    dict(ws=D), dict(T=1 << 27, V=1 << 28, ws_bytes=1 << 60), dict(T=64, D=512, ldx=512, ldw=512, ws_bytes=1 << 20),
])
def test_loss_refuses(kw):
    assert operators.load("linear_cross_entropy").linear_cross_entropy(*loss_args(**kw)) == INVALID


def loss_back_args(**kw):
    far = 1 << 40
    a = dict(dloss=A, X=B, W=C, target=D, saved=E, dX=F, dW=G, T=4, D=16, V=8, sg=1, ldx=16, ldw=16, st=1, lddx=16, lddw=16, type=0,
             ignore=-100, ws=far, ws_bytes=1 << 28, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(D=-1), dict(V=0), dict(T=(1 << 21) - 63), dict(V=1 << 31), dict(ldx=15), dict(ldw=15), dict(lddx=15), dict(lddw=15),
    dict(sg=-1), dict(st=-1), dict(type=2), dict(dloss=None), dict(X=None), dict(W=None), dict(target=None), dict(saved=None), dict(dX=None),
    dict(dW=None), dict(dloss=A + 2), dict(X=B + 1), dict(target=D + 4), dict(saved=E + 2), dict(dX=F + 1), dict(ws=None), dict(ws_bytes=64),
    dict(ws=(1 << 40) + 8), dict(dX=B), dict(dX=G), dict(dW=C), dict(dW=A), dict(dX=E), dict(ws=A), dict(ws=G),
])
def test_loss_backward_refuses(kw):
    assert operators.load("linear_cross_entropy").linear_cross_entropy_backward(*loss_back_args(**kw)) == INVALID


def test_loss_empty_and_workspace():
    lib = operators.load("linear_cross_entropy")
    assert lib.linear_cross_entropy(*loss_args(T=0, X=None, target=None, loss=None, ws=None, ws_bytes=0)) == 0
    assert lib.linear_cross_entropy_workspace(A, B, 0, 16, 8, 16, 16) == 0
    assert lib.linear_cross_entropy_workspace(A, B, 4, 16, 0, 16, 16) == -1
    plain_bytes = lib.linear_cross_entropy_workspace(A, B, 64, 64, 1000, 64, 64)
    assert 0 < plain_bytes < 1 << 20
    assert lib.linear_cross_entropy_workspace(A, B + 2, 64, 64, 1000, 64, 64) >= plain_bytes + 1000 * 64 * 2
    assert lib.linear_cross_entropy_workspace(A, B, 64, 63, 1000, 64, 64) >= plain_bytes + 1064 * 64 * 2
    assert lib.linear_cross_entropy_backward_workspace(A, B, 4, 16, 8, 16, 16) > 0
    assert lib.linear_cross_entropy_backward_workspace(A, B, 1 << 21, 16, 8, 16, 16) == -1
    # a piece of the vocabulary at a time: far below what the outputs would take
    T, D, V = 8192, 4096, 131072
    assert lib.linear_cross_entropy_workspace(A, B, T, D, V, D, D) < T * V // 4
    assert lib.linear_cross_entropy_backward_workspace(A, B, T, D, V, D, D) < T * V


@pytest.mark.parametrize("T", [0, 17, 64, 1000, 4096])
@pytest.mark.parametrize("D", [1032, 4096])
def test_loss_backward_workspace_holds_what_is_read(T, D):
    """Both images of dl and X transposed; W, which is read as it lies at these sizes, neither copied
    nor transposed (1 GB at 4096 x 131072); the parts of split sums, 32 MB."""
    V = 131072
    need = operators.load("linear_cross_entropy").linear_cross_entropy_backward_workspace(A, B, T, D, V, D, D)
    rows = (T + 63) // 64 * 64
    images = 2 * 2 * max(min(rows * V, 1 << 27), 1024 * rows) * 1.1  # (pieces are whole tiles)
    x = 2 * 2 * rows * (D + 64) + 4 * rows * (D + 64)  # whole lines, transposed; dX's sums
    assert need <= images + x + (36 << 20 if T else 4096)


def test_loss_bindings_refuse_host_tensors():
    x, w = torch.zeros(4, 16, dtype=torch.float16), torch.zeros(8, 16, dtype=torch.float16)
    target = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: fw.linear_cross_entropy(x, w, target), lambda: fw.linear_cross_entropy_train(x, w, target),
                 lambda: fw.linear_cross_entropy_backward(torch.zeros(4), x, w, target, torch.zeros(4, 3))):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [(5, 16, 40), (60, 72, 300)], ids=str)
def test_loss_bounds_reject_what_is_wrong(shape, t):
    """Zeros, a lost column of the vocabulary, a lost token, a one-hot that is missing, and gradients of another token's dloss."""
    T, D, V = shape
    t = plain.TYPES[t]
    gen = torch.Generator().manual_seed(V)
    x, w = torch.randn(T, D, generator=gen).to(t), (torch.randn(V, D, generator=gen) * D ** -0.5).to(t)
    target, g = torch.randint(0, V, (T,), generator=gen), torch.rand(T, generator=gen) + 0.1
    y, bound, parts = plain.loss(x, w, target)
    (dx, dw), (bx, bw) = plain.loss_gradients(g, t, parts)

    def outside(got, want, bound):
        return bool(((got - want).abs() > bound).any())

    for want, b in ((y, bound), (dx, bx), (dw, bw)):
        assert outside(torch.zeros_like(want), want, b)
    p, w64, x64 = parts[4], w.double(), x.double()
    assert outside(y + (1 - p[:, 0]).log(), y, bound)
    assert outside(dx - g.double()[:, None] * p[:, :1] * w64[:1], dx, bx)
    assert outside(dx + g.double()[:, None] * w64[target], dx, bx) and outside(dx.roll(1, 0), dx, bx)
    dl = g.double()[:, None] * (p - torch.nn.functional.one_hot(target, V))
    assert outside(dw - dl[:1].T @ x64[:1], dw, bw)


def test_plain_loss_gradients_match_differences():
    gen = torch.Generator().manual_seed(9)
    x, w = torch.randn(6, 5, generator=gen, dtype=torch.float64), torch.randn(11, 5, generator=gen, dtype=torch.float64)
    target = torch.tensor([0, 3, -100, 10, 3, 7])
    g = torch.randn(6, generator=gen, dtype=torch.float64)
    _, _, parts = plain.loss(x, w, target)
    grads, _ = plain.loss_gradients(g, torch.float16, parts)
    for i in range(2):
        v = torch.randn((x, w)[i].shape, generator=gen, dtype=torch.float64)
        ends = [(plain.loss(*(u + s * 1e-6 * v if k == i else u for k, u in enumerate((x, w))), target)[0] * g).sum() for s in (1, -1)]
        slope = float(ends[0] - ends[1]) / 2e-6
        assert abs(slope - float((grads[i] * v).sum())) <= 1e-6 * max(1.0, abs(slope))
