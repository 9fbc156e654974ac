"""The layer norm and its backward pass on an MI355X, through the public entry
points, against the 64-bit forms and bounds of ``_training``."""
from __future__ import annotations

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


def inputs(rows, cols, t, params, seed=0, mean=0.5):
    """x, weight, bias, dy"""
    x = normal(rows, cols, seed=seed, std=2.0) + mean
    return (x.to(t), (normal(cols, seed=seed + 1, std=0.2) + 1).to(params), normal(cols, seed=seed + 2, t=params),
            normal(rows, cols, seed=seed + 3, t=t))


def check(x, w, b, dy, y, saved, got, eps=1e-5, params=None):
    want, bound = plain.norm(x, w, b, eps)
    plain.assert_within(y, want, bound, "y")
    want, bounds = plain.norm_gradients(dy, x, w, eps, params)
    for name, g, v, e in zip(("dx", "dweight", "dbias"), got, want, bounds):
        if g is not None:
            plain.assert_within(g, v, e, name)


# below, at and past the widths at which a row takes more lanes or more chunks
# to a lane, for 16-bit (chunks of 8) and 32-bit elements (of 4); odd widths
SHAPES = [(1, 1), (5, 1), (3, 2), (7, 3), (70, 7), (33, 8), (9, 31), (64, 33), (130, 64), (65, 65), (31, 127), (40, 128), (41, 129),
          (10, 256), (11, 257), (200, 300), (9, 511), (8, 512), (5, 513), (100, 1000), (3, 1024), (6, 1025), (50, 1031), (2, 2048),
          (5, 2049), (700, 2731), (3, 4096), (2, 4097), (3, 5000), (300, 8192), (2, 8193), (5, 16384), (3, 16385), (2, 20001),
          (2, 32768), (2, 32775), (3, 70001)]


@pytest.mark.parametrize("t", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_gradients(shape, t):
    rows, cols = shape
    t = plain.TYPES[t]
    for params in {t, torch.float32}:
        x, w, b, dy = inputs(rows, cols, t, params, seed=rows + cols)
        y, saved = fw.layer_norm_train(x, w, b)
        assert torch.equal(y, fw.layer_norm(x, w, b))
        check(x, w, b, dy, y, saved, fw.layer_norm_backward(dy, x, w, b, saved))


@pytest.mark.parametrize("t", ["fp16", "fp32"])
@pytest.mark.parametrize("shape", [(20000, 64), (70000, 24), (9001, 200), (5000, 1000), (4100, 4096), (3000, 10000), (900, 40000), (70000, 13),
                                   (30000, 5), (9001, 201), (4100, 4095), (900, 16381)], ids=str)
def test_many_rows(shape, t):
    """More rows than the workgroups take at once."""
    x, w, b, dy = inputs(*shape, plain.TYPES[t], torch.float32, seed=3)
    y, saved = fw.layer_norm_train(x, w, b)
    check(x, w, b, dy, y, saved, fw.layer_norm_backward(dy, x, w, b, saved))


@pytest.mark.parametrize("shape", [(70, 600001), (5, 2 ** 22 + 4)], ids=str)
def test_columns_with_fewer_shares(shape):
    """Rows so long that fewer workgroups share them."""
    x, w, b, dy = inputs(*shape, torch.bfloat16, torch.float32, seed=4)
    y, saved = fw.layer_norm_train(x, w, b)
    check(x, w, b, dy, y, saved, fw.layer_norm_backward(dy, x, w, b, saved))


@pytest.mark.parametrize("cols", [40, 1000, 70000])
def test_without_parameters(cols):
    x, w, b, dy = inputs(30, cols, torch.bfloat16, torch.bfloat16)
    for weight, bias in ((None, None), (w, None), (None, b)):
        y, saved = fw.layer_norm_train(x, weight, bias, eps=1e-3)
        got = fw.layer_norm_backward(dy, x, weight, bias, saved)
        assert (got[1] is None) == (weight is None) and (got[2] is None) == (bias is None)
        check(x, weight, bias, dy, y, saved, got, 1e-3)


@pytest.mark.parametrize("cols", [50, 1000, 4096])
def test_rows_far_off_zero(cols):
    """A variance about the mean: a mean of a hundred deviations costs no digits but the mean's own."""
    x, w, b, dy = inputs(40, cols, torch.float32, torch.float32, mean=200.0)
    y, saved = fw.layer_norm_train(x, w, b)
    check(x, w, b, dy, y, saved, fw.layer_norm_backward(dy, x, w, b, saved))


def test_equal_elements():
    """No variance: eps alone; and one column, whose norm is the bias."""
    x = torch.full((5, 300), 3.0, dtype=torch.float16, device=DEV)
    w, b = normal(300, seed=1, t=torch.float16), normal(300, seed=2, t=torch.float16)
    y, saved = fw.layer_norm_train(x, w, b)
    assert torch.equal(y, b.expand(5, 300))
    dx, dw, db = fw.layer_norm_backward(x, x, w, b, saved)
    assert torch.isfinite(dx).all() and (dw == 0).all() and (db == 15).all()
    one = torch.randn(7, 1, device=DEV)
    y, saved = fw.layer_norm_train(one, w[:1].float(), b[:1].float())
    assert torch.equal(y, b[:1].float().expand(7, 1))
    assert (fw.layer_norm_backward(one, one, w[:1].float(), b[:1].float(), saved)[0] == 0).all()


@pytest.mark.parametrize("t", ["fp16", "fp32"])
@pytest.mark.parametrize("cols", [20, 700, 3001, 20000])
def test_gradients_match_differences(cols, t):
    """The 64-bit form's slope along random directions against the kernels' gradients."""
    x, w, b, dy = inputs(6, cols, plain.TYPES[t], plain.TYPES[t], seed=5)
    _, saved = fw.layer_norm_train(x, w, b)
    got = [v.double().cpu() for v in fw.layer_norm_backward(dy, x, w, b, saved)]
    _, bounds = plain.norm_gradients(dy, x, w)
    leaves = [v.double().cpu() for v in (x, w, b)]
    d64 = dy.double().cpu()

    def loss(x, w, b):
        c = x - x.mean(1, keepdim=True)
        return ((c / (c.square().mean(1, keepdim=True) + 1e-5).sqrt() * w + b) * d64).sum()

    for i in range(3):
        v = torch.randn(leaves[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        h = 1e-4
        ends = [loss(*(u + s * h * v if k == i else u for k, u in enumerate(leaves))) for s in (1, -1)]
        slope = float(ends[0] - ends[1]) / (2 * h)
        # (differences: third derivatives, of a value of order one per element, times h^2)
        assert abs(slope - float((got[i] * v).sum())) <= float((bounds[i] * v.abs()).sum()) + 1e-6 * (1 + abs(slope)) + 1e-6 * cols


@pytest.mark.parametrize("shape", [(40, 64), (9, 333), (20, 1000), (7, 4104), (3, 40000)], ids=str)
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_views_and_untouched_surroundings(shape, offset):
    x, w, b, dy = inputs(*shape, torch.bfloat16, torch.float32, seed=7)
    y, saved = fw.layer_norm_train(x, w, b)
    grads = fw.layer_norm_backward(dy, x, w, b, saved)
    vx, vdy = framed(x, offset=offset)[0], framed(dy, cols=5, offset=offset)[0]
    vy, big = framed(torch.zeros_like(x), offset=offset)
    out, s2 = fw.layer_norm_train(vx, w, b, out=vy)
    assert out is vy and torch.equal(vy, y) and torch.equal(s2, saved) and frame_intact(vy, big)
    vd, big = framed(torch.zeros_like(x), cols=3, offset=offset)
    wide = torch.full((2, shape[1] + 9), 7.0, device=DEV)
    got = fw.layer_norm_backward(vdy, vx, w, b, saved, out=(vd, wide[0, 1:1 + shape[1]], wide[1, 3:3 + shape[1]]))
    assert all(torch.equal(a, c) for a, c in zip(got, grads)) and frame_intact(vd, big)
    assert (wide[0, :1] == 7).all() and (wide[0, 1 + shape[1]:] == 7).all() and (wide[1, :3] == 7).all()


@pytest.mark.parametrize("cols", [24, 100, 1000, 5000, 50000])
def test_special_values_stay_in_their_rows(cols):
    x, w, b, dy = inputs(40, cols, torch.float16, torch.float16, seed=9)
    y, saved = fw.layer_norm_train(x, w, b)
    dx = fw.layer_norm_backward(dy, x, w, b, saved)[0]
    x[3, cols - 1], x[17, 0] = float("nan"), float("inf")
    bad, saved = fw.layer_norm_train(x, w, b)
    assert torch.isnan(bad[3]).all() and torch.isnan(bad[17]).all()
    keep = [r for r in range(40) if r not in (3, 17)]
    assert torch.equal(bad[keep], y[keep])
    got = fw.layer_norm_backward(dy, x, w, b, saved)[0]
    assert torch.isnan(got[3]).all() and torch.equal(got[keep], dx[keep])
    # an infinite gradient likewise, and a NaN in one weight reaches y's column alone
    dy[5, 1] = float("inf")
    x, w, b, _ = inputs(40, cols, torch.float16, torch.float16, seed=9)
    _, saved = fw.layer_norm_train(x, w, b)
    got = fw.layer_norm_backward(dy, x, w, b, saved)[0]
    assert not torch.isfinite(got[5]).any() and torch.equal(got[keep][:4], dx[keep][:4])
    w[2] = float("nan")
    one = fw.layer_norm(x, w, b)
    assert torch.isnan(one[:, 2]).all() and torch.equal(one[:, 3:], y[:, 3:])


def test_empty():
    t = torch.float16
    w = torch.ones(8, dtype=t, device=DEV)
    x = torch.zeros(0, 8, dtype=t, device=DEV)
    y, saved = fw.layer_norm_train(x, w, w)
    assert y.shape == (0, 8) and saved.shape == (0, 2)
    dx, dw, db = fw.layer_norm_backward(x, x, w, w, saved)
    assert dx.shape == (0, 8) and (dw == 0).all() and (db == 0).all()
    x, w = torch.zeros(4, 0, dtype=t, device=DEV), torch.ones(0, dtype=t, device=DEV)
    y, saved = fw.layer_norm_train(x, w, None)
    assert y.shape == (4, 0) and fw.layer_norm_backward(x, x, w, None, saved)[1].shape == (0,)


def test_past_32_bits():
    """More than 2^31 elements, and a pitch that takes the last row past 2^32 bytes."""
    rows, cols = 70000, 32768
    x = torch.empty(rows, cols, dtype=torch.float16, device=DEV).normal_()
    w = torch.ones(cols, device=DEV)
    y, saved = fw.layer_norm_train(x, w, None)
    at = torch.tensor([0, 65535, 65536, 69999])
    want, bound = plain.norm(x[at], w, None)
    plain.assert_within(y[at], want, bound)
    dx, dw, _ = fw.layer_norm_backward(x, x, w, None, saved)
    want, bounds = plain.norm_gradients(x[at], x[at], w)
    plain.assert_within(dx[at], want[0], bounds[0])
    # (dy = x: each of dweight's sums is of 70000 terms about 1)
    assert ((dw - rows).abs() < 0.05 * rows).all()
    del y, dx
    tall = x.reshape(7, -1)[:, 5:300]
    want, bound = plain.norm(tall, None, None)
    plain.assert_within(fw.layer_norm(tall), want, bound)


@pytest.mark.parametrize("shape", [(70000, 32768), (180000, 12000)], ids=str)
def test_sums_of_columns_past_32_bits(shape):
    """dweight and dbias of more than 2^31 elements, column by column: rows of any length, and held in registers."""
    rows, cols = shape
    x, w, b, dy = (torch.empty(*s, dtype=t, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(i)) for i, (s, t) in enumerate(
        ((shape, torch.float16), ((cols,), torch.float32), ((cols,), torch.float32), (shape, torch.float16))))
    _, saved = fw.layer_norm_train(x, w, b)
    _, dw, db = fw.layer_norm_backward(dy, x, w, b, saved)
    at = torch.tensor([0, 1, 7, 8, 2047, 2048, 4095, 8191, cols // 2 + 3, cols - 9, cols - 1], device=DEV)
    h, off = [], []
    for i in range(0, rows, 1000):
        parts = plain._norm_parts(x[i:i + 1000].double(), 1e-5)
        h.append(parts[0][:, at])
        off.append(parts[2][:, at])
    h, off, d = torch.cat(h), torch.cat(off), dy[:, at].double()
    # (the sums' additions as in plain.norm_gradients)
    adds = rows // 64 + 1 + 32 + 32 + 16 + 2
    want, bound = (d * h).sum(0), adds * plain.EPS * (d * h).abs().sum(0) + (d.abs() * off).sum(0)
    plain.assert_near(dw[at], want, bound + plain.rounded(want, torch.float32), "dweight")
    want, bound = d.sum(0), adds * plain.EPS * d.abs().sum(0)
    plain.assert_near(db[at], want, bound + plain.rounded(want, torch.float32), "dbias")


def test_refusals_on_gpu_tensors():
    x, w, b, dy = inputs(4, 16, torch.float16, torch.float16)
    y, saved = fw.layer_norm_train(x, w, b)
    for bad in (w[:8], w[None], w.bfloat16(), w.double(), w.cpu(), torch.ones(32, dtype=torch.float16, device=DEV)[::2]):
        with pytest.raises((TypeError, ValueError)):
            fw.layer_norm(x, bad, b)
    with pytest.raises(TypeError):
        fw.layer_norm(x, w, b.float())
    with pytest.raises(ValueError, match="eps"):
        fw.layer_norm(x, w, b, eps=-1.0)
    with pytest.raises(ValueError, match="eps"):
        fw.layer_norm(x, w, b, eps=float("nan"))
    with pytest.raises(fw.GemmError):
        fw.layer_norm(x, w, b, out=x)
    with pytest.raises(TypeError):
        fw.layer_norm(x, w, b, out=x.float())
    with pytest.raises(ValueError, match="saved"):
        fw.layer_norm_backward(dy, x, w, b, saved[:3])
    with pytest.raises(ValueError):
        fw.layer_norm_backward(dy[:3], x, w, b, saved)
    with pytest.raises(ValueError, match="dx, dweight and dbias"):
        fw.layer_norm_backward(dy, x, w, b, saved, out=(y,))
    with pytest.raises(ValueError, match="dbias"):
        fw.layer_norm_backward(dy, x, w, b, saved, out=(y, torch.empty_like(w), None))
    with pytest.raises(ValueError, match="dweight"):
        fw.layer_norm_backward(dy, x, None, b, saved, out=(y, torch.empty_like(w), torch.empty_like(b)))
    with pytest.raises(fw.GemmError):
        fw.layer_norm_backward(dy, x, w, b, saved, out=(dy, torch.empty_like(w), torch.empty_like(b)))
    same = torch.empty_like(w)
    with pytest.raises(fw.GemmError):
        fw.layer_norm_backward(dy, x, w, b, saved, out=(y, same, same))
