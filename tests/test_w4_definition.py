"""The 4-bit product at infinities, NaN and the ends of x's range: results are
those of the definition, sum over k of x * ((q - zero) * scale), and of their
signs, on every kernel."""
from __future__ import annotations

import pytest
import torch

import _operators as plain
import dense_fp16_gemm_04_amd as fw
from test_operators import DEV, _built, framed, w4_inputs  # noqa: F401

pytestmark = pytest.mark.gpu

# (M, N, K, group, offset of x): one and two blocks of 16 rows of W, one and two
# of x, tiles of 64 x 64 and 64 x 128, x off 16 bytes
SHAPES = [(1, 40, 256, 64, 0), (5, 33, 1056, 32, 0), (9, 8200, 288, 32, 0), (20, 40, 640, 128, 0), (40, 70, 320, 320, 0),
          (70, 5600, 288, 32, 0), (70, 8192, 256, 64, 0), (130, 4100, 384, 128, 0), (18, 50, 288, 32, 1)]


def defined(x, q, s, z):
    """The definition in 64 bits on the CPU, where no product or sum of these values overflows."""
    codes = plain.unpack(q)
    group = codes.shape[1] // s.shape[1]
    s = s.double().cpu().repeat_interleave(group, 1)
    z = torch.full_like(codes, 8.0) if z is None else z.double().cpu().repeat_interleave(group, 1)
    w = (codes - z) * s
    # (term by term: a library product may leave out what it multiplies by zero)
    return torch.stack([(row * w).sum(1) for row in x.double().cpu()])


def same_specials(got, want):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("zeros", [None, "whole", "any"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_w4_infinities_and_nan(shape, zeros, t):
    M, N, K, group, offset = shape
    x, q, s, z = w4_inputs(M, N, K, group, zeros, plain.TYPES[t], seed=sum(shape))
    clean = fw.gemv_w4(framed(x, offset=offset)[0], q, s, z)
    bad = {0: [(K - 1, float("inf"))]}
    if M > 8:
        bad[3] = [(0, float("-inf"))]
        bad[M - 1] = [(1, float("inf")), (K // 2, float("-inf"))]
        bad[5] = [(7, float("nan"))]
    rows = sorted(bad)
    for r in rows:
        for k, v in bad[r]:
            x[r, k] = v
    got = fw.gemv_w4(framed(x, offset=offset)[0], q, s, z)
    want = defined(x[rows], q, s, z)
    assert torch.isinf(want[0]).any()  # (codes that differ from their zero point)
    same_specials(got[rows], want)
    keep = [r for r in range(M) if r not in bad]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("zeros", [None, "whole"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_w4_large_finite_x(shape, zeros):
    """bfloat16 x whose sums with an offset of 128 leave the 32-bit range while results do not."""
    M, N, K, group, offset = shape
    x, q, s, z = w4_inputs(M, N, K, group, zeros, torch.bfloat16, seed=sum(shape))
    x = torch.randint(-1, 2, (M, K), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    x[:, 0] = 1.0
    x *= 2.0 ** 122
    s = (s.float() * 2.0 ** -8).bfloat16()
    want, bound = plain.product_w4(x, q, s, z)
    assert torch.isfinite(want).all()
    got = fw.gemv_w4(framed(x, offset=offset)[0], q, s, z)
    plain.assert_within(got, want, bound)


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_w4_infinite_scales_and_zeros(shape, t):
    M, N, K, group, offset = shape
    x, q, s, z = w4_inputs(M, N, K, group, "whole", plain.TYPES[t], seed=sum(shape))
    x[0, :group] = 0  # (times an infinite weight: NaN)
    s[3, 0] = float("inf")
    s[7, -1] = float("nan")
    z[11, 0] = float("inf")
    z[20, -1] = float("-inf")
    s[25, 0] = 0
    got = fw.gemv_w4(framed(x, offset=offset)[0], q, s, z)
    same_specials(got, defined(x, q, s, z))
