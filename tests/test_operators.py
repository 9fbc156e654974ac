"""The operators beside the product on an MI355X, through their public entry
points, against the 64-bit forms and bounds of ``_operators``."""
from __future__ import annotations

import os

import pytest
import torch

import _operators as plain
import dense_fp16_gemm_04_amd as fw
from dense_fp16_gemm_04_amd import build, operators

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not all(os.path.exists(operators.library_path(n)) for n in build.OPERATORS):
        import __graft_entry__
        __graft_entry__.build()


def normal(*shape, seed, std=1.0, t=torch.float32):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(t).to(DEV)


def framed(t, rows=2, cols=8, offset=0, fill=7.0):
    """A view holding t's values inside a larger buffer filled with `fill`, and the buffer."""
    big = torch.full((t.shape[0] + 2 * rows, t.shape[1] + 2 * cols + offset), fill, dtype=t.dtype, device=t.device)
    view = big[rows:rows + t.shape[0], cols + offset:cols + offset + t.shape[1]]
    view.copy_(t)
    return view, big


def frame_intact(view, big, fill=7.0):
    seen = big.clone()
    off = view.storage_offset()
    r, c = off // big.stride(0), off % big.stride(0)
    seen[r:r + view.shape[0], c:c + view.shape[1]] = fill
    return bool((seen == fill).all())


# ------------------------------------------------------------- gated_nt --

def gated_inputs(T, D, F, t, seed=0):
    return (normal(T, D, seed=seed, t=t), normal(F, D, seed=seed + 1, std=max(D, 1) ** -0.5, t=t),
            normal(F, D, seed=seed + 2, std=max(D, 1) ** -0.5, t=t))


# (T, D, F): single elements, one token, tails of every tile edge, odd widths
GATED_SHAPES = [(1, 1, 1), (1, 8, 1), (1, 64, 16), (1, 1024, 100), (2, 72, 33), (3, 200, 64), (7, 256, 130),
                (15, 136, 31), (16, 512, 48), (17, 64, 129), (33, 264, 65), (64, 128, 64), (65, 8, 257), (100, 33, 50),
                (128, 320, 128), (129, 640, 200), (255, 72, 70), (257, 1000, 129), (300, 65, 513)]


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("shape", GATED_SHAPES, ids=str)
def test_gated_forward_and_gradients(shape, act, t):
    T, D, F = shape
    t = plain.TYPES[t]
    x, wg, wu = gated_inputs(T, D, F, t, seed=sum(shape))
    h = fw.gated_nt(x, wg, wu, activation=act)
    want, bound = plain.gated(x, wg, wu, act)
    plain.assert_within(h, want, bound, "h")
    h2, saved = fw.gated_nt_train(x, wg, wu, activation=act)
    assert torch.equal(h, h2)
    dh = normal(T, F, seed=99, std=0.5, t=t)
    got = fw.gated_nt_backward(dh, x, wg, wu, saved)
    want, bounds = plain.gated_gradients(dh, x, wg, wu, act)
    for name, g, w, b in zip(("dx", "dw_gate", "dw_up"), got, want, bounds):
        plain.assert_within(g, w, b, name)


# up to 32 rows: K's steps of 64 dealt to eight waves, 8 or 16 columns of h
# to a workgroup
@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 4096, 24), (2, 2056, 4100), (5, 1000, 333), (8, 72, 8200), (9, 520, 40),
                                   (16, 8192, 130), (16, 1536, 4097), (13, 33, 5000), (4, 600, 1), (17, 4096, 100), (24, 200, 4100),
                                   (32, 1032, 331), (31, 8192, 9)], ids=str)
def test_gated_few_rows(shape, t):
    T, D, F = shape
    x, wg, wu = gated_inputs(T, D, F, plain.TYPES[t], seed=sum(shape))
    h, saved = fw.gated_nt_train(x, wg, wu, activation="gelu_tanh")
    want, bound = plain.gated(x, wg, wu, "gelu_tanh")
    plain.assert_within(h, want, bound, "h")
    assert torch.equal(h, fw.gated_nt(x, wg, wu, activation="gelu_tanh"))
    dh = normal(T, F, seed=37, t=plain.TYPES[t])
    got = fw.gated_nt_backward(dh, x, wg, wu, saved)
    want, bounds = plain.gated_gradients(dh, x, wg, wu, "gelu_tanh")
    for name, g, w, b in zip(("dx", "dw_gate", "dw_up"), got, want, bounds):
        plain.assert_within(g, w, b, name)
    for offset in (0, 1, 4):
        vh, big = framed(torch.zeros(T, F, dtype=plain.TYPES[t], device=DEV), offset=offset)
        fw.gated_nt(framed(x, offset=offset)[0], framed(wg, offset=offset)[0], wu, activation="gelu_tanh", out=vh)
        assert torch.equal(vh, h) and frame_intact(vh, big)


@pytest.mark.parametrize("shape", [(2048, 256, 4096), (4096, 520, 1000), (513, 1024, 2056)], ids=str)
def test_gated_many_tiles(shape):
    T, D, F = shape
    x, wg, wu = gated_inputs(T, D, F, torch.bfloat16, seed=5)
    h, saved = fw.gated_nt_train(x, wg, wu)
    want, bound = plain.gated(x, wg, wu, "silu")
    plain.assert_within(h, want, bound, "h")
    dh = normal(T, F, seed=6, std=0.1, t=torch.bfloat16)
    got = fw.gated_nt_backward(dh, x, wg, wu, saved)
    want, bounds = plain.gated_gradients(dh, x, wg, wu, "silu")
    for name, g, w, b in zip(("dx", "dw_gate", "dw_up"), got, want, bounds):
        plain.assert_within(g, w, b, name)


# more 256 x 256 tiles than CUs, and every way through their K loop: 3 to 17
# steps, whole and with a tail, so that tiles start at every ring position
@pytest.mark.parametrize("D", [136, 192, 200, 256, 320, 328, 448, 520, 640, 712, 1080])
@pytest.mark.parametrize("t", ["fp16", "bf16"])
def test_gated_tiles_in_turn(D, t):
    T, F = 256 * 18 + 5, 128 * 16 - 3
    x, wg, wu = gated_inputs(T, D, F, plain.TYPES[t], seed=D)
    h, saved = fw.gated_nt_train(x, wg, wu)
    want, bound = plain.gated(x, wg, wu, "silu")
    plain.assert_within(h, want, bound, "h")
    # the whole-piece stores of an output whose rows are a multiple of four
    plain.assert_within(fw.gated_nt(x, wg[:2040], wu[:2040]), want[:, :2040], bound[:, :2040], "whole pieces")


# sums so long (2F for dx, T for the weights) that the few tiles are split over
# K and joined; results with and without rows of eights
@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [(300, 296, 5001), (304, 301, 5000), (5003, 296, 136), (600, 1032, 2736)], ids=str)
def test_gated_long_sums(shape, t):
    T, D, F = shape
    x, wg, wu = gated_inputs(T, D, F, plain.TYPES[t], seed=7)
    h, saved = fw.gated_nt_train(x, wg, wu)
    want, bound = plain.gated(x, wg, wu, "silu")
    plain.assert_within(h, want, bound, "h")
    dh = normal(T, F, seed=8, std=0.1, t=plain.TYPES[t])
    got = fw.gated_nt_backward(dh, x, wg, wu, saved)
    want, bounds = plain.gated_gradients(dh, x, wg, wu, "silu")
    for name, g, w, b in zip(("dx", "dw_gate", "dw_up"), got, want, bounds):
        plain.assert_within(g, w, b, name)
    for g, again in zip(got, fw.gated_nt_backward(dh, x, wg, wu, saved)):
        assert torch.equal(g, again)


def test_gated_results_past_32_bits():
    """2.45e9 elements of h: offsets of rows, saved blocks and transposes."""
    T, D, F = 70000, 32, 35000
    t = torch.bfloat16
    x, wg, wu = gated_inputs(T, D, F, t, seed=9)
    h, saved = fw.gated_nt_train(x, wg, wu)
    rows, cols = torch.tensor([0, 61357, 69999]), torch.tensor([0, 1, 17501, 34999])
    want, bound = plain.gated(x[rows], wg, wu, "silu")
    plain.assert_within(h[rows], want, bound, "h")
    dh = torch.randn(T, F, dtype=t, device=DEV, generator=torch.Generator(DEV).manual_seed(10))
    dx, dwg, dwu = fw.gated_nt_backward(dh, x, wg, wu, saved)
    (want, _, _), (bound, _, _) = plain.gated_gradients(dh[rows], x[rows], wg, wu, "silu")
    plain.assert_within(dx[rows], want, bound, "dx")
    (_, *want), (_, *bound) = plain.gated_gradients(dh[:, cols], x, wg[cols], wu[cols], "silu")
    plain.assert_within(dwg[cols], want[0], bound[0], "dw_gate")
    plain.assert_within(dwu[cols], want[1], bound[1], "dw_up")


@pytest.mark.parametrize("t", ["fp16", "bf16"])
def test_gated_infinite_weights_do_not_meet_the_padding(t):
    """One infinite weight: act(g) = +inf in its column, and so is the gradient
    of w_up's row; NaN would be zeros past the last token times that weight."""
    T, D, F = 5, 16, 20
    t = plain.TYPES[t]
    x, wg, wu = gated_inputs(T, D, F, t, seed=33)
    x = x.abs() + 0.25
    dh = normal(T, F, seed=36, t=t).abs() + 0.25
    _, saved = fw.gated_nt_train(x, wg, wu)
    clean = fw.gated_nt_backward(dh, x, wg, wu, saved)
    bad = wg.clone()
    bad[3, 0] = float("inf")
    _, saved = fw.gated_nt_train(x, bad, wu)
    _, dwg, dwu = fw.gated_nt_backward(dh, x, bad, wu, saved)
    assert (dwu[3] == float("inf")).all()
    keep = [r for r in range(F) if r != 3]
    assert torch.equal(dwu[keep], clean[2][keep]) and torch.equal(dwg[keep], clean[1][keep])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_gradients_match_differences(act):
    T, D, F = 37, 72, 50
    t = torch.float16
    x, wg, wu = gated_inputs(T, D, F, t, seed=40)
    dh = normal(T, F, seed=43, std=0.5, t=t)
    _, saved = fw.gated_nt_train(x, wg, wu, activation=act)
    got = fw.gated_nt_backward(dh, x, wg, wu, saved)
    _, bounds = plain.gated_gradients(dh, x, wg, wu, act)
    leaves = [v.double().cpu() for v in (x, wg, wu)]
    d64 = dh.double().cpu()

    def loss(a, b, c):
        return (plain.activation(a @ b.T, act)[0] * (a @ c.T) * d64).sum()

    for i in range(3):
        v = torch.randn(leaves[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        step = 1e-5
        plus, minus = ([w + s * step * v if k == i else w for k, w in enumerate(leaves)] for s in (1, -1))
        difference = float((loss(*plus) - loss(*minus)) / (2 * step))
        have = float((got[i].double().cpu() * v).sum())
        # the elements' bounds along v, and the difference's own error
        assert abs(have - difference) <= float((bounds[i] * v.abs()).sum()) + 1e-6 * (1 + abs(difference))


@pytest.mark.parametrize("offset", [0, 1, 4])
def test_gated_views_and_untouched_surroundings(offset):
    """Operands and results inside larger buffers: rows apart, 16-byte aligned or not."""
    T, D, F = 70, 72, 90
    t = torch.float16
    x, wg, wu = gated_inputs(T, D, F, t, seed=11)
    dh = normal(T, F, seed=12, t=t)
    vx, vg, vu, vd = (framed(v, offset=offset)[0] for v in (x, wg, wu, dh))
    h_ref, saved_ref = fw.gated_nt_train(x, wg, wu)
    ref = fw.gated_nt_backward(dh, x, wg, wu, saved_ref)
    vh, big_h = framed(torch.zeros(T, F, dtype=t, device=DEV), offset=offset)
    out, saved = fw.gated_nt_train(vx, vg, vu, out=vh)
    assert out is vh and torch.equal(vh, h_ref) and frame_intact(vh, big_h)
    assert torch.equal(fw.gated_nt(vx, vg, vu), h_ref)
    outs = [framed(torch.zeros(*s, dtype=t, device=DEV), offset=offset) for s in ((T, D), (F, D), (F, D))]
    got = fw.gated_nt_backward(vd, vx, vg, vu, saved, out=[v for v, _ in outs])
    for g, r, (v, big) in zip(got, ref, outs):
        assert g is v and torch.equal(v, r) and frame_intact(v, big)


def test_gated_weights_with_unlike_pitches():
    x, wg, wu = gated_inputs(40, 64, 48, torch.bfloat16, seed=21)
    vg, vu = framed(wg, cols=8)[0], framed(wu, cols=16)[0]
    assert vg.stride(0) != vu.stride(0)
    assert torch.equal(fw.gated_nt(x, vg, vu), fw.gated_nt(x, wg, wu))


def test_gated_halves_of_one_weight():
    """w_gate and w_up as the two halves of one [2F, D] weight."""
    x, wg, wu = gated_inputs(40, 64, 48, torch.bfloat16, seed=22)
    both = torch.cat((wg, wu))
    assert torch.equal(fw.gated_nt(x, both[:48], both[48:]), fw.gated_nt(x, wg, wu))


def test_gated_same_weight_twice():
    x, wg, _ = gated_inputs(40, 64, 48, torch.float16, seed=23)
    want, bound = plain.gated(x, wg, wg, "silu")
    plain.assert_within(fw.gated_nt(x, wg, wg), want, bound)


@pytest.mark.parametrize("shape", [(0, 16, 8), (4, 16, 0), (4, 0, 8), (0, 0, 0), (0, 16, 300)], ids=str)
def test_gated_empty(shape):
    T, D, F = shape
    x, wg, wu = gated_inputs(T, D, F, torch.float16)
    h, saved = fw.gated_nt_train(x, wg, wu)
    assert h.shape == (T, F) and (h == 0).all()
    ones = torch.full((T + F + 1, max(D, 1)), 3.0, dtype=torch.float16, device=DEV)
    outs = [ones[:T, :D].clone(), ones[:F, :D].clone(), ones[:F, :D].clone()]
    dx, dwg, dwu = fw.gated_nt_backward(torch.zeros(T, F, dtype=torch.float16, device=DEV), x, wg, wu, saved, out=outs)
    assert dx.shape == (T, D) and dwg.shape == dwu.shape == (F, D)
    assert (dx == 0).all() and (dwg == 0).all() and (dwu == 0).all()


@pytest.mark.parametrize("t", ["fp16", "bf16"])
def test_gated_special_values_stay_in_their_rows(t):
    t = plain.TYPES[t]
    T, D, F = 40, 72, 70
    x, wg, wu = gated_inputs(T, D, F, t, seed=31)
    clean, _ = fw.gated_nt_train(x, wg, wu)
    bad = x.clone()
    bad[3, 5] = float("inf")
    bad[9, 0] = float("nan")
    bad[20, 71] = float("-inf")
    got, _ = fw.gated_nt_train(bad, wg, wu)
    for r in range(T):
        if r in (3, 20):
            # +-inf * weight: +inf (or nan) where act(+inf) * u, 0 * inf = nan where g -> -inf
            want, _ = plain.gated(bad[r:r + 1], wg, wu, "silu")
            assert torch.equal(torch.isnan(got[r].cpu()), torch.isnan(want[0]))
        elif r == 9:
            assert torch.isnan(got[r]).all()
        else:
            assert torch.equal(got[r], clean[r])
    # large inputs saturate the activation without NaN
    big = torch.full((2, 8), 100.0, dtype=t, device=DEV)
    w = torch.ones(4, 8, dtype=t, device=DEV)
    neg = fw.gated_nt(big, -w, w)
    assert (neg == 0).all()


def test_gated_overflow_is_infinite():
    x = torch.full((1, 64), 30000.0, dtype=torch.float16, device=DEV)
    w = torch.ones(16, 64, dtype=torch.float16, device=DEV)
    assert torch.isinf(fw.gated_nt(x, w, w)).all()


# ----------------------------------------------------- orthogonalize_ns --

NS_SHAPES = [(1, 1), (1, 9), (5, 1), (3, 4), (8, 8), (17, 16), (16, 33), (64, 64), (65, 63), (100, 300), (130, 128),
             (257, 100), (320, 320), (64, 1000), (700, 130)]


def ns_close(got, g, **kw):
    """Against the iteration with the documented roundings: a bfloat16
    rounding (half a step, 2^-8 of each value) and what single steps of
    binary16, taken the other way because a 32-bit sum is off by 2^-20, add up
    to (an entry in a hundred, by 2^-11, amplified by less than 10: 2^-10)."""
    want = plain.newton_schulz(g, rounded=True, **kw)
    err = (got.double().cpu() - want).norm(dim=(-2, -1))
    assert (err <= (2.0 ** -8 + 2.0 ** -10) * want.norm(dim=(-2, -1))).all(), (err, want.norm(dim=(-2, -1)))
    return want


@pytest.mark.parametrize("t", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("shape", NS_SHAPES, ids=str)
def test_ns(shape, t):
    g = normal(*shape, seed=sum(shape), std=0.01, t=plain.TYPES[t])
    out = fw.orthogonalize_ns(g)
    assert out.dtype == torch.bfloat16 and out.shape == g.shape
    want = ns_close(out, g)
    # and the documented roundings themselves: under 1% of the exact iteration
    # for a matrix of noise (steps of 2^-11, fifteen of them, amplified by less than 10 each)
    exact = plain.newton_schulz(g)
    assert (want - exact).norm() <= 15 * 10 * 2.0 ** -11 / 8 * exact.norm()


@pytest.mark.parametrize("shape", [(3, 65, 100), (5, 130, 70), (2, 256, 256), (7, 1, 3)], ids=str)
def test_ns_batch_equals_its_matrices(shape):
    g = normal(*shape, seed=4, t=torch.bfloat16)
    out = fw.orthogonalize_ns(g)
    ns_close(out, g)
    for i in range(shape[0]):
        assert torch.equal(out[i], fw.orthogonalize_ns(g[i]))


@pytest.mark.parametrize("shape", [(2, 1030, 1536), (6, 1537, 1030), (9, 1024, 1280), (40, 516, 520)], ids=str)
def test_ns_large_tiles(shape):
    """Tiles of every size, more of them than CUs, with tails and without."""
    g = normal(*shape, seed=8, t=torch.bfloat16)
    out = fw.orthogonalize_ns(g, steps=2)
    ns_close(out[:2], g[:2], steps=2)
    ns_close(out[-1], g[-1], steps=2)


@pytest.mark.parametrize("shape", [(300, 9000), (9001, 203), (2, 520, 6000), (1100, 2900)], ids=str)
def test_ns_long_sums(shape):
    """Few tiles of long sums, split over K and joined."""
    g = normal(*shape, seed=12, t=torch.bfloat16)
    out = fw.orthogonalize_ns(g, steps=3)
    ns_close(out, g, steps=3)
    assert torch.equal(out, fw.orthogonalize_ns(g, steps=3))


@pytest.mark.parametrize("shape", [(20000, 256, 512), (5000, 64, 8192)], ids=str)
def test_ns_batch_past_32_bits(shape):
    """2.6e9 elements in all."""
    g = torch.randn(*shape, dtype=torch.bfloat16, device=DEV, generator=torch.Generator(DEV).manual_seed(13))
    out = fw.orthogonalize_ns(g, steps=2)
    for i in (0, shape[0] * 5 // 6, shape[0] - 1):
        ns_close(out[i], g[i], steps=2)


@pytest.mark.parametrize("t", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("shape", [(64, 4096), (50, 8192), (8192, 33), (64, 8193), (8200, 64), (1, 5000), (7, 129),
                                   (193, 64), (63, 1025), (2, 64, 64), (3, 1279, 17)], ids=str)
def test_ns_few_rows(shape, t):
    """Sixty-four rows or fewer: one to all chunks of columns, one to many workgroups."""
    g = normal(*shape, seed=14, std=0.02, t=plain.TYPES[t])
    out = fw.orthogonalize_ns(g)
    ns_close(out, g)
    assert torch.equal(out, fw.orthogonalize_ns(g))
    ns_close(fw.orthogonalize_ns(g, steps=1), g, steps=1)
    ns_close(fw.orthogonalize_ns(g, steps=0), g, steps=0)


@pytest.mark.parametrize("shape", [(40, 333), (333, 40), (64, 128)], ids=str)
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_ns_few_rows_in_views(shape, offset):
    g = normal(*shape, seed=15, t=torch.float16)
    ref = fw.orthogonalize_ns(g)
    vo, big = framed(torch.zeros(shape, dtype=torch.bfloat16, device=DEV), offset=offset)
    assert fw.orthogonalize_ns(framed(g, offset=offset)[0], out=vo) is vo
    assert torch.equal(vo, ref) and frame_intact(vo, big)
    wide = torch.stack((g, -g, 2 * g, g))
    wide[1, 3, 3] = float("nan")
    out = fw.orthogonalize_ns(wide)
    assert torch.equal(out[0], ref) and torch.equal(out[3], ref) and torch.isnan(out[1]).all()


def test_ns_small_diagonals_of_the_polynomial():
    """Diagonal entries of P of every size: 0, below binary16's range, ordinary."""
    g = torch.eye(24, 40, device=DEV) * torch.linspace(0.05, 1.0, 24, device=DEV)[:, None]
    s = g.double().cpu()
    s = (s / s.norm()).square().sum(1)  # S is diagonal, and so is P: a + b s + c s s
    for a in (0.0, -float(s[10]), 1e-7, 3.0):
        ns_close(fw.orthogonalize_ns(g, steps=1, coefficients=(a, 1.0, 0.0)), g, steps=1, coefficients=(a, 1.0, 0.0))


def test_ns_steps_and_coefficients():
    g = normal(40, 70, seed=5)
    for steps in (0, 1, 2, 7):
        ns_close(fw.orthogonalize_ns(g, steps=steps), g, steps=steps)
    per_step = [(4.0, -6.0, 3.0), (3.0, -3.5, 1.5), (1.875, -1.25, 0.375)]
    ns_close(fw.orthogonalize_ns(g, steps=3, coefficients=per_step), g, steps=3, coefficients=per_step)
    ns_close(fw.orthogonalize_ns(g, eps=10.0), g, eps=10.0)


@pytest.mark.parametrize("scale", [1e-30, 1e-10, 1e10, 1e30])
def test_ns_does_not_depend_on_the_scale(scale):
    """Squares of these entries leave the 32-bit range."""
    g = normal(33, 50, seed=6)
    ns_close(fw.orthogonalize_ns(g * scale, eps=0.0), g * scale, eps=0.0)


def test_ns_rank_one_and_zero():
    u, v = normal(60, 1, seed=1), normal(1, 90, seed=2)
    ns_close(fw.orthogonalize_ns(u @ v), u @ v)
    e = torch.zeros(60, 90, device=DEV)
    e[3, 4] = 5.0
    ns_close(fw.orthogonalize_ns(e), e)
    assert (fw.orthogonalize_ns(torch.zeros(20, 30, device=DEV)) == 0).all()


def test_ns_special_values_stay_in_their_matrix():
    g = normal(3, 40, 50, seed=9, t=torch.bfloat16)
    clean = fw.orthogonalize_ns(g)
    bad = g.clone()
    bad[1, 2, 3] = float("nan")
    out = fw.orthogonalize_ns(bad)
    assert torch.isnan(out[1]).all()
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
    bad[1, 2, 3] = float("inf")
    assert torch.isnan(fw.orthogonalize_ns(bad)[1]).any()


@pytest.mark.parametrize("shape", [(70, 50), (50, 70), (64, 64)], ids=str)
@pytest.mark.parametrize("offset", [0, 1])
def test_ns_views(shape, offset):
    g = normal(*shape, seed=10, t=torch.bfloat16)
    ref = fw.orthogonalize_ns(g)
    vg = framed(g, offset=offset)[0]
    vo, big = framed(torch.zeros(shape, dtype=torch.bfloat16, device=DEV), offset=offset)
    assert fw.orthogonalize_ns(vg, out=vo) is vo
    assert torch.equal(vo, ref) and frame_intact(vo, big)
    # a batch whose matrices lie between others, and one matrix repeated
    wide = torch.stack((g, -g, 2 * g, g))
    out = fw.orthogonalize_ns(wide[::2])
    assert torch.equal(out[0], ref)
    same = fw.orthogonalize_ns(g.expand(3, *shape))
    assert all(torch.equal(s, ref) for s in same)


def test_ns_empty():
    for s in ((0, 5), (5, 0), (0, 5, 6), (2, 0, 3)):
        out = fw.orthogonalize_ns(torch.zeros(s, device=DEV))
        assert out.shape == s and out.dtype == torch.bfloat16


# -------------------------------------------------------------- gemv_w4 --

def w4_inputs(M, N, K, group, zeros, t, seed=0):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (N, K // 2), generator=gen, dtype=torch.uint8).to(DEV)
    groups = K // group if K else 0
    scales = (torch.rand(N, groups, generator=gen) * 0.1 + 0.01).to(t).to(DEV)
    z = None
    if zeros == "whole":
        z = torch.randint(0, 16, (N, groups), generator=gen).to(t).to(DEV)
    elif zeros == "any":
        z = (torch.rand(N, groups, generator=gen) * 20 - 2).to(t).to(DEV)
    return normal(M, K, seed=seed + 1, t=t), q, scales, z


W4_SHAPES = [(1, 1, 32, 32), (1, 16, 64, 32), (1, 17, 128, 64), (1, 100, 256, 128), (2, 33, 96, 32), (3, 15, 160, 32),
             (1, 64, 1024, 1024), (5, 40, 96, 96), (16, 48, 192, 64), (17, 16, 384, 128), (31, 50, 2048, 256),
             (33, 18, 1056, 32), (64, 32, 640, 128), (65, 7, 288, 32), (200, 70, 512, 64), (1, 40, 32, 32),
             (4, 20, 4160, 64)]


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("zeros", [None, "whole", "any"])
@pytest.mark.parametrize("shape", W4_SHAPES, ids=str)
def test_w4(shape, zeros, t):
    M, N, K, group = shape
    x, q, s, z = w4_inputs(M, N, K, group, zeros, plain.TYPES[t], seed=sum(shape))
    got = fw.gemv_w4(x, q, s, z)
    want, bound = plain.product_w4(x, q, s, z)
    plain.assert_within(got, want, bound)


# results of 512 tiles of 32 x 32 and more, for which 64 rows of x are taken at
# a time (by 64 of w, or 128 where binary16 has no zero points); K below, at
# and past whole blocks of 256
W4_MANY = [(33, 8200, 288, 32), (64, 8192, 512, 64), (70, 5600, 32, 32), (129, 4100, 480, 480), (200, 2400, 1280, 128),
           (513, 3650, 96, 32), (520, 3700, 704, 64), (1030, 2049, 256, 256)]


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("zeros", [None, "any"])
@pytest.mark.parametrize("shape", W4_MANY, ids=str)
def test_w4_many_rows(shape, zeros, t):
    M, N, K, group = shape
    x, q, s, z = w4_inputs(M, N, K, group, zeros, plain.TYPES[t], seed=sum(shape))
    got = fw.gemv_w4(x, q, s, z)
    want, bound = plain.product_w4(x, q, s, z)
    plain.assert_within(got, want, bound)
    assert torch.equal(got, fw.gemv_w4(x, q, s, z))


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("zeros", [None, "whole"])
def test_w4_many_rows_in_views(zeros, offset):
    """Rows and results inside larger buffers; a NaN and an infinity stay in their rows."""
    x, q, s, z = w4_inputs(150, 4101, 320, 64, zeros, torch.float16, seed=6)
    x[5, 7] = float("nan")
    x[149, 319] = float("inf")
    ref = fw.gemv_w4(x, q, s, z)
    assert torch.isnan(ref[5]).all() and not torch.isfinite(ref[149]).any()
    keep = [r for r in range(150) if r not in (5, 149)]
    want, bound = plain.product_w4(x[keep], q, s, z)
    plain.assert_within(ref[keep], want, bound)
    vy, big = framed(torch.zeros_like(ref), offset=offset)
    fw.gemv_w4(framed(x)[0], q, s, z, out=vy)
    assert torch.equal(vy[keep], ref[keep]) and frame_intact(vy, big)
    # (x off 16 bytes: another kernel, the same bounds)
    plain.assert_within(fw.gemv_w4(framed(x, offset=1)[0], q, s, z)[keep], want, bound)


def test_w4_results_past_32_bits():
    M, N, K = 70000, 35000, 32
    x, q, s, z = w4_inputs(M, N, K, 32, "whole", torch.float16, seed=7)
    rows = torch.tensor([0, 61357, 69999])
    want, bound = plain.product_w4(x[rows], q, s, z)
    plain.assert_within(fw.gemv_w4(x, q, s, z)[rows], want, bound)


@pytest.mark.parametrize("t", ["fp16", "bf16"])
def test_w4_every_code_in_every_place(t):
    """One-hot rows of x read single weights back."""
    t = plain.TYPES[t]
    K = 256
    codes = torch.stack([(torch.arange(K) + i) % 16 for i in range(16)])
    x = torch.eye(K, dtype=t, device=DEV)
    s = torch.full((16, K // 32), 0.5, dtype=t, device=DEV)
    got = fw.gemv_w4(x, plain.pack(codes).to(DEV), s)
    assert torch.equal(got.double().cpu(), (codes.double() - 8).T * 0.5)
    z = torch.full((16, K // 32), 3.0, dtype=t, device=DEV)
    got = fw.gemv_w4(x, plain.pack(codes).to(DEV), s, z)
    assert torch.equal(got.double().cpu(), (codes.double() - 3).T * 0.5)


def test_w4_views_and_untouched_surroundings():
    x, q, s, z = w4_inputs(9, 40, 256, 64, "any", torch.float16, seed=3)
    ref = fw.gemv_w4(x, q, s, z)
    for offset in (0, 1):
        vx = framed(x, offset=offset)[0]
        vy, big = framed(torch.zeros_like(ref), offset=offset)
        assert fw.gemv_w4(vx, q, s, z, out=vy) is vy
        assert torch.equal(vy, ref) and frame_intact(vy, big)
    wide = torch.zeros(40, 256, dtype=torch.uint8, device=DEV)
    wide[:, 32:160] = q
    assert torch.equal(fw.gemv_w4(x, wide[:, 32:160], s, z), ref)
    with pytest.raises(ValueError, match="16 bytes"):
        fw.gemv_w4(x, framed(q, cols=1)[0], s, z)


def test_w4_special_values_stay_in_their_rows():
    for zeros in (None, "whole"):
        x, q, s, z = w4_inputs(20, 40, 256, 64, zeros, torch.bfloat16, seed=4)
        ref = fw.gemv_w4(x, q, s, z)
        x[3, 7] = float("nan")
        x[17, 200] = float("inf")
        got = fw.gemv_w4(x, q, s, z)
        assert torch.isnan(got[3]).all() and not torch.isfinite(got[17]).any()
        keep = [r for r in range(20) if r not in (3, 17)]
        assert torch.equal(got[keep], ref[keep])


def test_w4_rows_do_not_depend_on_each_other():
    """A row's result is the same alone and among others."""
    x, q, s, z = w4_inputs(70, 40, 512, 128, "whole", torch.float16, seed=5)
    y = fw.gemv_w4(x, q, s, z)
    for r in (0, 16, 69):
        assert torch.equal(fw.gemv_w4(x[r:r + 1], q, s, z)[0], y[r])


def test_w4_empty():
    t = torch.float16
    q = torch.zeros(8, 0, dtype=torch.uint8, device=DEV)
    x, s = torch.zeros(3, 0, dtype=t, device=DEV), torch.zeros(8, 0, dtype=t, device=DEV)
    assert (fw.gemv_w4(x, q, s, out=torch.ones(3, 8, dtype=t, device=DEV)) == 0).all()
    x, q, s, _ = w4_inputs(3, 8, 64, 32, None, t)
    assert fw.gemv_w4(x[:0], q, s).shape == (0, 8)
    assert fw.gemv_w4(x, q[:0], s[:0]).shape == (3, 0)


def test_w4_bad_groups():
    x, q, s, _ = w4_inputs(3, 8, 192, 96, None, torch.float16)
    with pytest.raises(ValueError, match="power of two"):
        fw.gemv_w4(x, q, s)
    with pytest.raises(ValueError):
        fw.gemv_w4(x, q, s[:, :0])


# ------------------------------------------------- streams, graphs, both --

def everything(x, wg, wu, dh, q, s):
    h, saved = fw.gated_nt_train(x, wg, wu)
    dx, dwg, dwu = fw.gated_nt_backward(dh, x, wg, wu, saved)
    return [h, dx, dwg, dwu, fw.orthogonalize_ns(dwg), fw.orthogonalize_ns(torch.stack((dwg, dwu))), fw.gemv_w4(x, q, s)]


def everything_inputs(seed, T=96):
    x, wg, wu = gated_inputs(T, 256, 320, torch.float16, seed=seed)
    dh = normal(T, 320, seed=seed + 5, t=torch.float16)
    _, q, s, _ = w4_inputs(1, 200, 256, 64, None, torch.float16, seed=seed)
    return [x, wg, wu, dh, q, s]


def test_results_repeat_bit_for_bit():
    args = everything_inputs(50)
    first = everything(*args)
    for _ in range(3):
        for a, b in zip(first, everything(*args)):
            assert torch.equal(a, b)


def test_streams_side_by_side():
    sets = [everything_inputs(60 + i, T=64 + 32 * i) for i in range(3)]
    want = [everything(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None] * len(sets)
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = everything(*sets[i])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for a, b in zip(w, g):
            assert torch.equal(a, b)


def test_captured_graphs_replay():
    """Two graphs of all operators, replayed in turn on changing inputs with
    eager work between, against eager results."""
    sets = [everything_inputs(70), everything_inputs(80, T=33)]
    graphs, outs = [], []
    for args in sets:
        everything(*args)  # libraries loaded, allocator warm
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(everything(*args))
        graphs.append(g)
    for k in range(4):
        for args, g, out in zip(sets, graphs, outs):
            for i, v in enumerate(everything_inputs(100 + k, T=args[0].shape[0])):
                args[i].copy_(v)
            g.replay()
            torch.cuda.synchronize()
            kept = [o.clone() for o in out]
            for a, b in zip(kept, everything(*args)):
                assert torch.equal(a, b)


def small_calls(x, wg, wu, g, tall, q, s, xs):
    """The kernels of few rows: decoding, small updates, and a prompt in 4 bits."""
    return [fw.gated_nt(x, wg, wu), fw.gated_nt(x[:3], wg, wu), fw.orthogonalize_ns(g), fw.orthogonalize_ns(tall),
            fw.gemv_w4(xs, q, s), fw.gemv_w4(xs[:9], q, s)]


def small_inputs(seed, T=20):
    x, wg, wu = gated_inputs(T, 1160, 515, torch.bfloat16, seed=seed)
    _, q, s, _ = w4_inputs(1, 8200, 288, 32, None, torch.float16, seed=seed)
    return [x, wg, wu, normal(3, 40, 777, seed=seed + 6), normal(900, 64, seed=seed + 7, t=torch.float16), q, s,
            normal(70, 288, seed=seed + 8, t=torch.float16)]


def test_small_calls_on_streams_and_in_graphs():
    sets = [small_inputs(110), small_inputs(120, T=32)]
    want = [small_calls(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None] * len(sets)
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = small_calls(*sets[i])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))
    graphs, outs = [], []
    for args in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(small_calls(*args))
        graphs.append(g)
    for k in range(4):
        for args, g, out in zip(sets, graphs, outs):
            for i, v in enumerate(small_inputs(130 + k, T=args[0].shape[0])):
                args[i].copy_(v)
            g.replay()
            torch.cuda.synchronize()
            kept = [o.clone() for o in out]
            assert all(torch.equal(a, b) for a, b in zip(kept, small_calls(*args)))


@pytest.mark.parametrize("T", [1, 4, 16, 29])
def test_gated_few_rows_keep_special_values_to_themselves(T):
    x, wg, wu = gated_inputs(T, 600, 300, torch.float16, seed=38)
    clean = fw.gated_nt(x, wg, wu)
    bad = x.clone()
    bad[T - 1, 599] = float("nan")
    got = fw.gated_nt(bad, wg, wu)
    assert torch.isnan(got[T - 1]).all() and torch.equal(got[:T - 1], clean[:T - 1])
    heavy = wg.clone()
    heavy[299, 0] = float("inf")
    got = fw.gated_nt(x, heavy, wu)
    assert torch.equal(got[:, :299], clean[:, :299]) and not torch.isfinite(got[x[:, 0] > 0, 299]).any()


def test_on_another_current_device(monkeypatch):
    """The operand's device is entered when another one is current (simulated on one GPU)."""
    args = everything_inputs(90)
    want = everything(*args)
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
    got = [fw.gated_nt(*args[:3]), fw.gemv_w4(args[0], args[4], args[5])]
    monkeypatch.undo()
    assert entered == [0, 0]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[6])


def test_refusals_on_gpu_tensors():
    x, wg, wu = gated_inputs(4, 16, 8, torch.float16)
    _, saved = fw.gated_nt_train(x, wg, wu)
    dh = torch.zeros(4, 8, dtype=torch.float16, device=DEV)
    with pytest.raises(ValueError, match="activation"):
        fw.gated_nt(x, wg, wu, activation="tanh")
    with pytest.raises(TypeError):
        fw.gated_nt(x, wg.bfloat16(), wu)
    with pytest.raises(ValueError):
        fw.gated_nt(x, wg, wu[:7])
    with pytest.raises(ValueError):
        fw.gated_nt(x[:, :8], wg, wu)
    with pytest.raises(ValueError):
        fw.gated_nt(x.T.contiguous().T, wg, wu)
    with pytest.raises(ValueError):
        fw.gated_nt(x[:1].expand(4, 16), wg, wu)
    with pytest.raises(ValueError):
        fw.gated_nt(x, wg, wu, out=dh[:, :7])
    with pytest.raises(fw.GemmError):
        fw.gated_nt(x, wg, wu, out=x[:, :8])
    with pytest.raises(ValueError, match="saved"):
        fw.gated_nt_backward(dh, x, wg, wu, saved[:-1])
    with pytest.raises(ValueError):
        fw.gated_nt_backward(dh[:3], x, wg, wu, saved)
    with pytest.raises(ValueError, match="three"):
        fw.gated_nt_backward(dh, x, wg, wu, saved, out=[x])
    with pytest.raises(fw.GemmError):
        fw.gated_nt_backward(dh, x, wg, wu, saved, out=[x, wg.clone(), wu.clone()])
    with pytest.raises(TypeError):
        fw.orthogonalize_ns(wg, out=wg)
    with pytest.raises(fw.GemmError):
        same = wg.bfloat16()
        fw.orthogonalize_ns(same, out=same)
    with pytest.raises(ValueError, match="overlap"):
        fw.orthogonalize_ns(torch.zeros(2, 8, 16, device=DEV),
                            out=torch.zeros(8, 16, dtype=torch.bfloat16, device=DEV).expand(2, 8, 16))


def test_a_layer_trained_updated_and_served():
    """The operators as they are used together: a feed-forward block's forward
    and backward pass around the library's product, its weights' updates
    orthogonalised, and the updated weight served in 4 bits."""
    T, D, F = 200, 128, 192
    t = torch.float16
    x, wg, wu = gated_inputs(T, D, F, t, seed=200)
    wd = normal(D, F, seed=203, std=F ** -0.5, t=t)
    target = normal(T, D, seed=204, t=t)
    h, saved = fw.gated_nt_train(x, wg, wu)
    y = fw.gemm_nt_f16(h, wd)
    dy = ((y.float() - target.float()) * 0.01).to(t)
    dh = fw.gemm_nt_f16(dy, wd.t().contiguous())
    dx, dwg, dwu = fw.gated_nt_backward(dh, x, wg, wu, saved)
    want, bounds = plain.gated_gradients(dh, x, wg, wu, "silu")
    for g, w, b in zip((dx, dwg, dwu), want, bounds):
        plain.assert_within(g, w, b)
    update = fw.orthogonalize_ns(torch.stack((dwg, dwu)))
    ns_close(update, torch.stack((dwg, dwu)))
    new = (wg.float() - 0.02 * update[0].float())
    # four bits and a scale per 64 weights, codes about 8
    blocks = new.reshape(F, D // 64, 64)
    s = (blocks.abs().amax(-1) / 7).to(t)
    codes = (blocks / s.float()[..., None]).round().clamp(-8, 7) + 8
    q = plain.pack(codes.reshape(F, D).cpu()).to(DEV)
    one = x[:1]
    got = fw.gemv_w4(one, q, s)
    want, bound = plain.product_w4(one, q, s, None)
    plain.assert_within(got, want, bound)
    # and the quantised layer is the updated one within its own step: half a
    # code (and the clamp's none) per weight
    exact = one.double().cpu() @ new.double().cpu().T
    step = one.double().cpu().abs() @ s.double().cpu().repeat_interleave(64, 1).T
    assert ((got.double().cpu() - exact).abs() <= 0.51 * step + bound).all()
