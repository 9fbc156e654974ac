"""The loss over a vocabulary and its gradients on an MI355X, through the public
entry points, against the 64-bit forms and bounds of ``_training``."""
from __future__ import annotations

import math
import os

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


def inputs(T, D, V, t, seed=0, ignored=0.2, sure=4.0):
    """x, w, target, dloss: some tokens foreseen, some ignored."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    w = (normal(V, D) * max(D, 1) ** -0.5).to(t)
    target = torch.randint(0, V, (T,), generator=gen, device=DEV)
    x = (normal(T, D) + sure * torch.rand(T, 1, generator=gen, device=DEV) * w.float()[target]).to(t)
    target[torch.rand(T, generator=gen, device=DEV) < ignored] = -100
    return x, w, target, normal(T) / max(T, 1)


def check(x, w, target, dloss, loss, got, ignore=-100):
    want, bound, parts = plain.loss(x, w, target, ignore)
    plain.assert_near(loss, want, bound, "loss")
    want, bounds = plain.loss_gradients(dloss, x.dtype, parts, rounded=len(x) > 16)
    for name, g, v, b in zip(("dx", "dw"), got, want, bounds):
        plain.assert_near(g, v, b, name)


def step(x, w, target, dloss, **kw):
    loss, saved = fw.linear_cross_entropy_train(x, w, target, **kw)
    return loss, fw.linear_cross_entropy_backward(dloss, x, w, target, saved, **kw)


# (T, D, V): single elements, one token, tails of every tile edge, odd widths
SHAPES = [(1, 1, 1), (1, 8, 1), (1, 64, 5), (2, 3, 2), (3, 72, 33), (1, 256, 4000), (7, 130, 999), (8, 1, 70), (16, 512, 65), (17, 64, 129),
          (33, 264, 1000), (64, 128, 64), (65, 136, 257), (100, 33, 1000), (129, 64, 129), (255, 8, 300), (257, 1000, 129), (300, 65, 513),
          (40, 1000, 3001), (511, 520, 770)]


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_loss_and_gradients(shape, t):
    x, w, target, dloss = inputs(*shape, plain.TYPES[t], seed=sum(shape))
    loss, got = step(x, w, target, dloss)
    assert torch.equal(loss, fw.linear_cross_entropy(x, w, target))
    check(x, w, target, dloss, loss, got)


# up to 16 tokens: with 1, 4, 8 and 16 rows of registers; one and several pieces
# of D; vocabularies below and above where more rows of w go to a workgroup, and
# that no share or block divides; odd widths and D below a step
@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1030, 33), (2, 7, 4097), (3, 4100, 70), (4, 31, 25000), (5, 2049, 515), (8, 333, 30001), (9, 1025, 66),
                                   (12, 65, 24577), (13, 3491, 1001), (16, 2056, 131), (16, 520, 40000), (15, 4096, 3)], ids=str)
def test_few_tokens(shape, t):
    x, w, target, dloss = inputs(*shape, plain.TYPES[t], seed=sum(shape))
    loss, got = step(x, w, target, dloss)
    assert torch.equal(loss, fw.linear_cross_entropy(x, w, target))
    check(x, w, target, dloss, loss, got)
    # (the same in views at other addresses, bit for bit)
    vx, vw = framed(x, cols=3, offset=1)[0], framed(w, cols=5)[0]
    l2, (dx, dw) = step(vx, vw, target, dloss)
    assert torch.equal(l2, loss) and torch.equal(dx, got[0]) and torch.equal(dw, got[1])


# the largest tiles, more of them than CUs, with tails; and K loops of 3 to 17
# steps, whole and with a tail, so that tiles start at every ring position
@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [(4101, D, 4093) for D in (136, 192, 200, 256, 320, 328, 520, 712, 1080)] +
                         [(2048, 264, 9001), (1000, 1032, 8003), (5000, 72, 16400)], ids=str)
def test_many_tiles(shape, t):
    x, w, target, dloss = inputs(*shape, plain.TYPES[t], seed=sum(shape))
    loss, got = step(x, w, target, dloss)
    check(x, w, target, dloss, loss, got)


@pytest.mark.parametrize("shape", [(300, 2048, 300), (64, 8200, 500), (513, 4104, 257), (2500, 200, 200)], ids=str)
def test_sums_in_parts(shape):
    """Few tiles of long sums, over D, over the vocabulary, over the tokens."""
    x, w, target, dloss = inputs(*shape, torch.float16, seed=4)
    loss, got = step(x, w, target, dloss)
    check(x, w, target, dloss, loss, got)


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [(9000, 136, 33001), (20000, 64, 16500), (140000, 24, 3000)], ids=str)
def test_pieces_of_the_vocabulary(shape, t):
    """More than 2^27 outputs: dx adds up over pieces, the last one odd."""
    x, w, target, dloss = inputs(*shape, plain.TYPES[t], seed=5)
    loss, got = step(x, w, target, dloss)
    check(x, w, target, dloss, loss, got)


# long sums over the vocabulary, which dx's product takes from w as it lies: in place
# and copied, over vocabularies and to widths that no step, tile or part divides,
# rows that span more than 32 bits, and two pieces of the vocabulary
@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [(17, 4096, 20001), (200, 1000, 9001), (129, 520, 20007), (600, 1160, 30002), (200, 333, 30001)], ids=str)
def test_w_as_it_lies(shape, t):
    x, w, target, dloss = inputs(*shape, plain.TYPES[t], seed=sum(shape))
    loss, got = step(x, w, target, dloss)
    check(x, w, target, dloss, loss, got)
    # (between its rows and behind them there may be anything)
    vw = framed(w, cols=24, offset=8)[0]
    l2, (dx, dw) = step(x, vw, target, dloss)
    assert torch.equal(l2, loss) and torch.equal(dx, got[0]) and torch.equal(dw, got[1])


def test_large_products():
    """X is copied to whole lines, or lies in them: the same bits."""
    x, w, target, dloss = inputs(4100, 1000, 16001, torch.bfloat16, seed=22)
    loss, got = step(x, w, target, dloss)
    check(x, w, target, dloss, loss, got)
    lines = torch.full((4100, 1024), float("nan"), dtype=torch.bfloat16, device=DEV)[:, :1000]
    lines.copy_(x)
    l2, (dx, dw) = step(lines, w, target, dloss)
    assert torch.equal(l2, loss) and torch.equal(dx, got[0]) and torch.equal(dw, got[1])


def test_w_far_apart():
    T, D, V = 200, 1000, 20000
    x, w, target, dloss = inputs(T, D, V, torch.float16, seed=20)
    far = torch.empty(V, 1 << 17, dtype=torch.float16, device=DEV)[:, :D]
    far.copy_(w)
    loss, got = step(x, w, target, dloss)
    l2, (dx, dw) = step(x, far, target, dloss)
    assert torch.equal(l2, loss) and torch.equal(dx, got[0]) and torch.equal(dw, got[1])


@pytest.mark.parametrize("shape", [(40, 776, 2 ** 20 + 5003)], ids=str)
def test_w_as_it_lies_in_pieces(shape):
    x, w, target, dloss = inputs(*shape, torch.bfloat16, seed=21)
    loss, got = step(x, w, target, dloss)
    check(x, w, target, dloss, loss, got)


@pytest.mark.parametrize("shape", [(1, 24, 2 ** 20 + 70), (3, 8, 2 ** 21 + 5)], ids=str)
def test_vocabularies_past_a_pitch(shape):
    x, w, target, dloss = inputs(*shape, torch.bfloat16, seed=6, ignored=0.0)
    loss, got = step(x, w, target, dloss)
    check(x, w, target, dloss, loss, got)


def test_outputs_past_32_bits():
    """T times V past 2^32, targets at the far end."""
    T, D, V = 40000, 16, 110000
    x, w, target, dloss = inputs(T, D, V, torch.float16, seed=7)
    target[-1], target[0] = V - 1, 0
    loss, (dx, dw) = step(x, w, target, dloss)
    rows = torch.tensor([0, 1, 20000, T - 2, T - 1], device=DEV)
    want, bound, parts = plain.loss(x[rows], w, target[rows])
    plain.assert_near(loss[rows], want, bound)
    want, bounds = plain.loss_gradients(dloss[rows], x.dtype, parts)
    plain.assert_near(dx[rows], want[0], bounds[0])
    # dw's sum over the vocabulary: the rows of dl add up to 0
    mean = dw.double().mean(0)
    assert (mean.abs() <= 1e-3 * dw.double().abs().mean(0)).all()


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [(5, 40, 70), (300, 136, 513), (4101, 200, 4093)], ids=str)
def test_near_certain_tokens(shape, t):
    """Probabilities next to 1 and 0: losses down to nothing, 1 - p without cancellation in the type."""
    x, w, target, dloss = inputs(*shape, plain.TYPES[t], seed=8, ignored=0.0, sure=0.0)
    x = (w.float()[target] * torch.linspace(0, 60, shape[0], device=DEV)[:, None] * 1.0 + x.float() * 0.2).to(x.dtype)
    loss, got = step(x, w, target, dloss)
    assert (loss >= 0).all()
    check(x, w, target, dloss, loss, got)


@pytest.mark.parametrize("scale", [1e-12, 1e-6, 1.0, 1e4])
@pytest.mark.parametrize("t", ["fp16", "bf16"])
def test_gradients_of_any_size(scale, t):
    """dloss is followed by a power of two in binary16; dw's own type ends where it ends."""
    x, w, target, dloss = inputs(130, 72, 333, plain.TYPES[t], seed=9)
    dloss = dloss * scale
    loss, got = step(x, w, target, dloss)
    check(x, w, target, dloss, loss, got)


@pytest.mark.parametrize("shape", [(70, 64, 200), (4101, 136, 4093)], ids=str)
def test_large_and_low_outputs(shape):
    """Outputs of hundreds, all far below zero (columns that are not there may not show), and of one row all alike."""
    T, D, V = shape
    x, w, target, dloss = inputs(T, D, V, torch.bfloat16, seed=10)
    for shift in (-40.0, 40.0):
        ws = w.clone()
        ws[:, 0] = shift
        xs = x.clone()
        xs[:, 0] = 8.0
        loss, got = step(xs, ws, target, dloss)
        check(xs, ws, target, dloss, loss, got)
    xs = x.clone()
    xs[3] = 0
    loss, got = step(xs, w, target, dloss)
    check(xs, w, target, dloss, loss, got)
    assert target[3] < 0 or abs(float(loss[3]) - math.log(V)) < 1e-5


@pytest.mark.parametrize("t", ["fp16", "bf16"])
def test_gradients_match_differences(t):
    x, w, target, dloss = inputs(40, 72, 150, plain.TYPES[t], seed=11)
    _, got = step(x, w, target, dloss)
    _, _, parts = plain.loss(x, w, target)
    _, bounds = plain.loss_gradients(dloss, x.dtype, parts)
    leaves = [x.double(), w.double()]
    valid = target != -100
    at = torch.where(valid, target, torch.zeros_like(target))[:, None]

    def total(x, w):
        l = x @ w.T
        return ((torch.logsumexp(l, 1) - l.gather(1, at)[:, 0]) * valid * dloss.double()).sum()

    for i in range(2):
        v = normal(*leaves[i].shape, seed=20 + i).double()
        h = 1e-5
        ends = [total(*(u + s * h * v if k == i else u for k, u in enumerate(leaves))) for s in (1, -1)]
        slope = float(ends[0] - ends[1]) / (2 * h)
        assert abs(slope - float((got[i].double() * v).sum())) <= float((bounds[i] * v.abs()).sum()) + 1e-7 * (1 + abs(slope))


@pytest.mark.parametrize("shape", [(40, 72, 130), (5, 33, 70), (300, 136, 1000)], ids=str)
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_views_and_untouched_surroundings(shape, offset):
    T, D, V = shape
    x, w, target, dloss = inputs(*shape, torch.float16, seed=12)
    loss, saved = fw.linear_cross_entropy_train(x, w, target)
    dx, dw = fw.linear_cross_entropy_backward(dloss, x, w, target, saved)
    vx, vw = framed(x, offset=offset)[0], framed(w, cols=5, offset=offset)[0]
    wide = torch.zeros(T, 3, dtype=torch.int64, device=DEV)
    wide[:, 1] = target
    vl = torch.full((T + 2,), 7.0, device=DEV)
    out, s2 = fw.linear_cross_entropy_train(vx, vw, wide[:, 1], out=vl[1:-1])
    assert torch.equal(out, loss) and torch.equal(s2, saved) and vl[0] == 7 and vl[-1] == 7
    vdx, bx = framed(torch.zeros_like(x), offset=offset)
    vdw, bw = framed(torch.zeros_like(w), cols=3, offset=offset)
    g = torch.zeros(T, 2, device=DEV)
    g[:, 0] = dloss
    got = fw.linear_cross_entropy_backward(g[:, 0], vx, vw, wide[:, 1], saved, out=(vdx, vdw))
    assert got[0] is vdx and torch.equal(vdx, dx) and torch.equal(vdw, dw) and frame_intact(vdx, bx) and frame_intact(vdw, bw)


def test_one_gradient_for_all_tokens():
    """dloss expanded from one number, as the gradient of a sum is."""
    x, w, target, _ = inputs(70, 64, 100, torch.bfloat16, seed=13)
    _, saved = fw.linear_cross_entropy_train(x, w, target)
    one = torch.full((1,), 0.25, device=DEV)
    got = fw.linear_cross_entropy_backward(one.expand(70), x, w, target, saved)
    want = fw.linear_cross_entropy_backward(torch.full((70,), 0.25, device=DEV), x, w, target, saved)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("shape", [(6, 64, 100), (300, 136, 1000), (4101, 136, 4093)], ids=str)
@pytest.mark.parametrize("t", ["fp16", "bf16"])
def test_ignored_tokens_leave_no_trace(shape, t):
    """NaN and infinities in their rows, and in their dloss; all tokens ignored."""
    T, D, V = shape
    x, w, target, dloss = inputs(*shape, plain.TYPES[t], seed=14, ignored=0.5)
    target[1], target[0] = -100, 3
    loss, got = step(x, w, target, dloss)
    gone = target == -100
    assert (loss[gone] == 0).all() and (got[0][gone] == 0).all()
    for v in (float("nan"), float("inf"), -1e4):
        bad, g = x.clone(), dloss.clone()
        bad[gone], g[gone] = v, v
        bad[1, ::2] *= -1
        l2, g2 = step(bad, w, target, g)
        assert torch.equal(l2, loss) and all(torch.equal(a, b) for a, b in zip(g2, got))
    none = torch.full_like(target, 7 if V > 7 else 0)
    l2, g2 = step(x, w, none, dloss, ignore_index=int(none[0]))
    assert (l2 == 0).all() and all((v == 0).all() for v in g2)


def test_other_ignore_indices():
    x, w, target, dloss = inputs(50, 64, 90, torch.float16, seed=15)
    loss, got = step(x, w, target, dloss)
    for index in (0, 89, -1, 1 << 40):
        moved = torch.where(target == -100, torch.full_like(target, index), target)
        loss, got = step(x, w, moved, dloss, ignore_index=index)
        check(x, w, moved, dloss, loss, got, index)


def test_targets_outside_the_vocabulary():
    """NaN in the token's loss and its row of dx, and in dw."""
    x, w, target, dloss = inputs(70, 64, 100, torch.float16, seed=16)
    target[2] = 5
    loss, (dx, _) = step(x, w, target, dloss)
    for bad in (100, 101, -1, -99, 1 << 33, (1 << 32) + 5, -(1 << 62)):
        t2 = target.clone()
        t2[2] = bad
        l2, (dx2, dw2) = step(x, w, t2, dloss)
        keep = torch.arange(70, device=DEV) != 2
        assert torch.isnan(l2[2]) and torch.equal(l2[keep], loss[keep])
        assert torch.isnan(dx2[2]).all() and torch.equal(dx2[keep], dx[keep]) and torch.isnan(dw2).all()


@pytest.mark.parametrize("shape", [(30, 64, 100), (300, 136, 1000), (4101, 136, 4093)], ids=str)
def test_special_values_stay_in_their_rows(shape):
    T, D, V = shape
    x, w, target, dloss = inputs(*shape, torch.bfloat16, seed=17, ignored=0.0)
    loss, (dx, _) = step(x, w, target, dloss)
    bad = x.clone()
    bad[3, D - 1], bad[17, 0] = float("nan"), float("inf")
    l2, (dx2, _) = step(bad, w, target, dloss)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[3] = keep[17] = False
    assert torch.isnan(l2[3]) and not torch.isfinite(l2[17])
    assert torch.equal(l2[keep], loss[keep]) and torch.equal(dx2[keep], dx[keep])
    assert torch.isnan(dx2[3]).all() and not torch.isfinite(dx2[17]).all()
    # a row of w that leaves a token no probability there: exp(-infinity) is 0
    low = w.clone()
    low[V - 1] = 0
    low[V - 1, 0] = float("-inf")
    pos = x.clone()
    pos[:, 0] = pos[:, 0].abs() + 0.5
    t2 = torch.where(target == V - 1, torch.zeros_like(target), target)
    l2, (dx2, dw2) = step(pos, low, t2, dloss)
    want, _ = step(pos, w[:V - 1].contiguous(), t2, dloss)
    assert torch.allclose(l2, want, rtol=1e-5, atol=1e-5) and (dw2[V - 1] == 0).all()


# up to 16 tokens (D with and without a last chunk that ends with it, in the first round
# of loads and behind whole ones) and more
@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [(2, 7, 50), (3, 12, 70), (16, 33, 100), (5, 1033, 130), (8, 1033, 25000), (1, 1040, 66), (17, 33, 100),
                                   (40, 1033, 130)], ids=str)
def test_one_infinite_weight(shape, t):
    """Minus infinity in each of the last sixteen columns of a row of w, which leaves that row no
    probability: losses and gradients are those of the rows without it."""
    T, D, V = shape
    x, w, target, dloss = inputs(*shape, plain.TYPES[t], seed=24)
    target = torch.where(target == V - 1, torch.zeros_like(target), target)
    for c in range(max(0, D - 16), D):
        pos, low = x.clone(), w.clone()
        pos[:, c] = pos[:, c].abs() + 0.5
        low[V - 1, c] = float("-inf")
        loss, (dx, dw) = step(pos, low, target, dloss)
        want, bound, parts = plain.loss(pos, w[:V - 1], target)
        plain.assert_near(loss, want, bound, "loss, column %d" % c)
        want, bounds = plain.loss_gradients(dloss, x.dtype, parts, rounded=T > 16)
        rest = torch.arange(D, device=DEV) != c  # (column c of dx is 0 times the infinity)
        plain.assert_near(dx[:, rest], want[0][:, rest], bounds[0][:, rest], "dx, column %d" % c)
        plain.assert_near(dw[:V - 1], want[1], bounds[1], "dw, column %d" % c)
        assert (dw[V - 1] == 0).all()


@pytest.mark.parametrize("shape", [(0, 16, 8), (4, 0, 8), (0, 0, 5), (0, 16, 3000)], ids=str)
def test_empty(shape):
    T, D, V = shape
    x, w, target, dloss = inputs(*shape, torch.float16, ignored=0.0)
    loss, (dx, dw) = step(x, w, target, dloss)
    assert loss.shape == (T,) and dx.shape == (T, D) and dw.shape == (V, D) and (dw == 0).all()
    assert ((loss - math.log(V)).abs() < 1e-6).all()


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [(17, 0, 8), (300, 0, 513), (5000, 0, 40)], ids=str)
def test_no_columns(shape, t):
    """D of 0 above 16 tokens: every output is zero."""
    T, D, V = shape
    x, w, target, dloss = inputs(*shape, plain.TYPES[t])
    loss, saved = fw.linear_cross_entropy_train(x, w, target)
    dx, dw = fw.linear_cross_entropy_backward(dloss, x, w, target, saved)
    valid = target != -100
    assert ((loss - math.log(V))[valid].abs() < 1e-6 * math.log(V)).all() and (loss[~valid] == 0).all()
    assert dx.shape == (T, 0) and dw.shape == (V, 0)
    assert torch.equal(saved[valid], torch.tensor([0.0, V, 0.0], device=DEV).expand(int(valid.sum()), 3))


def some_rows_of_dw(x, w, target, dloss, rows, chunk):
    """(dw[rows], bound) by plain.loss_gradients, the tokens `chunk` at a time."""
    kept = []
    for i in range(0, len(x), chunk):
        part = slice(i, i + chunk)
        xc, w64, valid, at, p, l, top, s, s_rel, l_off = plain.loss(x[part], w, target[part])[2]
        here = at == rows
        # (a column more, for the targets that are not among `rows`)
        at = torch.where(here.any(1, keepdim=True), here.int().argmax(1, keepdim=True), torch.full_like(at, len(rows)))
        wide = [torch.cat([v[:, rows], torch.zeros_like(v[:, :1])], 1) for v in (p, l, l_off)]
        kept.append((xc, valid, at, wide[0], wide[1], top, s, s_rel, wide[2]))
    xc, valid, at, p, l, top, s, s_rel, l_off = (torch.cat(v) for v in zip(*kept))
    w64 = torch.cat([w[rows], w[:1]]).double()
    want, bounds = plain.loss_gradients(dloss, x.dtype, (xc, w64, valid, at, p, l, top, s, s_rel, l_off), rounded=len(x) > 16)
    return want[1][:-1], bounds[1][:-1]


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape, piece", [((40000, 16, 110000), 3584), ((9000, 136, 33001), 11008)], ids=str)
def test_rows_of_dw_in_pieces_of_the_vocabulary(shape, piece, t):
    """Outputs past 32 bits and pieces of the vocabulary: dw on both sides of pieces' ends, of targets and of both ends."""
    T, D, V = shape
    x, w, target, dloss = inputs(*shape, plain.TYPES[t], seed=25)
    target[-1], target[0] = V - 1, 0
    _, (_, dw) = step(x, w, target, dloss)
    ends = [v for e in range(piece, V, piece) for v in (e - 1, e)]
    rows = torch.tensor(sorted({0, 1, V - 2, V - 1, *ends, *target[target >= 0][:20].tolist()}), device=DEV)
    want, bound = some_rows_of_dw(x, w, target, dloss, rows, 2000)
    plain.assert_near(dw[rows], want, bound, "dw")


@pytest.mark.parametrize("shape", [(2100, 136, 2100), (2100, 133, 2100), (9, 136, 2100)], ids=str)
def test_gradients_that_lie_far_apart(shape):
    """dx and dw whose last rows lie past 2^32 bytes."""
    T, D, V = shape
    x, w, target, dloss = inputs(*shape, torch.bfloat16, seed=26)
    _, saved = fw.linear_cross_entropy_train(x, w, target)
    want = fw.linear_cross_entropy_backward(dloss, x, w, target, saved)
    far = [torch.full((n, 1 << 20), 7.0, dtype=x.dtype, device=DEV) for n in (T, V)]
    got = fw.linear_cross_entropy_backward(dloss, x, w, target, saved, out=[f[:, 8:8 + D] for f in far])
    for g, f, v in zip(got, far, want):
        assert torch.equal(g, v) and (f[:, :8] == 7).all() and (f[:, 8 + D:] == 7).all()


def test_refusals_on_gpu_tensors():
    x, w, target, dloss = inputs(4, 16, 8, torch.float16)
    loss, saved = fw.linear_cross_entropy_train(x, w, target)
    for bad in (target.int(), target.float(), [1, 2, 3, 4]):
        with pytest.raises(TypeError, match="target"):
            fw.linear_cross_entropy(x, w, bad)
    for bad in (target[:3], target[:, None], target.cpu()):
        with pytest.raises(ValueError, match="target"):
            fw.linear_cross_entropy(x, w, bad)
    with pytest.raises(TypeError):
        fw.linear_cross_entropy(x, w.bfloat16(), target)
    with pytest.raises(TypeError):
        fw.linear_cross_entropy(x.float(), w.float(), target)
    with pytest.raises(ValueError):
        fw.linear_cross_entropy(x, w[:, :8], target)
    with pytest.raises(ValueError):
        fw.linear_cross_entropy(x, w[:0], target)
    with pytest.raises(TypeError):
        fw.linear_cross_entropy(x, w, target, out=loss.half())
    for bad in (1 << 63, -(1 << 63) - 1):
        with pytest.raises(ValueError, match="ignore_index"):
            fw.linear_cross_entropy(x, w, target, ignore_index=bad)
        with pytest.raises(ValueError, match="ignore_index"):
            fw.linear_cross_entropy_backward(dloss, x, w, target, saved, ignore_index=bad)
    with pytest.raises(ValueError, match="saved"):
        fw.linear_cross_entropy_backward(dloss, x, w, target, saved[:3])
    with pytest.raises(ValueError, match="dloss"):
        fw.linear_cross_entropy_backward(dloss[:3], x, w, target, saved)
    with pytest.raises(TypeError, match="dloss"):
        fw.linear_cross_entropy_backward(dloss.half(), x, w, target, saved)
    with pytest.raises(ValueError, match="two matrices"):
        fw.linear_cross_entropy_backward(dloss, x, w, target, saved, out=(x,))
    with pytest.raises(fw.GemmError):
        fw.linear_cross_entropy_backward(dloss, x, w, target, saved, out=(x, torch.empty_like(w)))
    with pytest.raises(fw.GemmError):
        fw.linear_cross_entropy_backward(dloss, x, w, target, saved, out=(torch.empty_like(x), w))
