"""Plain 64-bit forms of the operators beside the product, and bounds on how
far a correct kernel may be from them (test infrastructure).

Each bound adds what the operator's documentation allows:
* a rounding to the result's type: half a step, finfo.eps / 2 of the value
  (and half of the type's smallest step, for subnormals);
* a 32-bit sum of n terms: n * 2^-23 of the sum of the terms' magnitudes (each
  addition off by at most a whole step, so that truncation is covered too);
* exp2, rcp and the few products after them: 2^-19 of the value.
"""
from __future__ import annotations

import math

import numpy as np
import torch

SUM = 2.0 ** -23
FUN = 2.0 ** -19
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def half_step(t):
    """(relative, absolute) error of one rounding to type t."""
    i = torch.finfo(t)
    return i.eps / 2, i.smallest_normal * i.eps / 2


def activation(g, act):
    """act(g), act'(g) in 64 bits, from the functions' textbook forms."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    k = math.sqrt(2 / math.pi)
    th = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * k * (1 + 3 * 0.044715 * g * g)


def gated(x, wg, wu, act):
    """(h, bound of h's error) for a kernel that sums in 32 bits."""
    t = x.dtype
    x, wg, wu = (v.double().cpu() for v in (x, wg, wu))
    g, u = x @ wg.T, x @ wu.T
    a, _ = activation(g, act)
    h = a * u
    dg, du = gated_sums_error(x, wg), gated_sums_error(x, wu)
    rel, absolute = half_step(t)
    # |act'| <= 1.13
    bound = 1.13 * u.abs() * dg + a.abs() * du + 1.13 * dg * du + (FUN + rel) * h.abs() + absolute
    return h, bound


def gated_sums_error(x, w):
    return SUM * (x.shape[1] + 1) * (x.abs() @ w.abs().T)


def gated_gradients(dh, x, wg, wu, act):
    """((dx, dwg, dwu), their bounds)."""
    t = x.dtype
    dh, x, wg, wu = (v.double().cpu() for v in (dh, x, wg, wu))
    T, F = dh.shape
    g, u = x @ wg.T, x @ wu.T
    eg, eu = gated_sums_error(x, wg), gated_sums_error(x, wu)
    a, da = activation(g, act)
    dg, du = dh * u * da, dh * a
    rel, absolute = half_step(t)
    # |act''| <= 0.8, |act'| <= 1.13
    p_err = 0.8 * u.abs() * eg + 1.13 * eu + 0.8 * eg * eu + FUN * (1 + g.abs()) * u.abs()
    q_err = 1.13 * eg + FUN * a.abs()
    dg_err = dh.abs() * p_err * (1 + rel) + rel * dg.abs() + absolute
    du_err = dh.abs() * q_err * (1 + rel) + rel * du.abs() + absolute
    dx = dg @ wg + du @ wu
    mag = (dg.abs() + dg_err) @ wg.abs() + (du.abs() + du_err) @ wu.abs()
    dx_b = dg_err @ wg.abs() + du_err @ wu.abs() + SUM * (2 * F + 1) * mag + rel * dx.abs() + absolute
    out, bounds = [dx], [dx_b * (1 + rel)]
    for d, e in ((dg, dg_err), (du, du_err)):
        dw = d.T @ x
        b = e.T @ x.abs() + SUM * (T + 1) * ((d.abs() + e).T @ x.abs()) + rel * dw.abs() + absolute
        out.append(dw)
        bounds.append(b * (1 + rel))
    return out, bounds


def newton_schulz(g, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, rounded=False):
    """The iteration in 64 bits; `rounded`: with X, S and the polynomial
    rounded to binary16 where the operator's documentation holds them so (X
    times the power of two nearest sqrt(longer side), rows times what rounding
    took from the polynomial's diagonal)."""
    x = g.double().cpu()
    if x.dim() == 3:
        return torch.stack([newton_schulz(v, steps, coefficients, eps, rounded) for v in x])
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    scale = 2.0 ** min(12, round(0.5 * math.log2(x.shape[1]))) if rounded else 1.0
    r = (lambda v, s=1.0: (v * s).half().double() / s) if rounded else (lambda v, s=1.0: v)
    x = r(x / (x.norm() + eps), scale)
    for k in range(steps):
        a, b, c = coefficients[k] if hasattr(coefficients[0], "__len__") else coefficients
        s = r(x @ x.T)
        p = a * torch.eye(len(s), dtype=torch.float64) + b * s + c * (s @ s)
        x = r(p) @ x
        if rounded:
            d, d16 = p.diagonal(), r(p).diagonal()
            x = x * torch.where(d16.abs() >= 2.0 ** -14, d / d16, torch.ones_like(d))[:, None]
        if k + 1 < steps:
            x = r(x, scale)
    return x.T if tall else x


def unpack(q):
    """Codes [N, K] of packed bytes [N, K / 2]."""
    q = q.cpu().numpy()
    out = np.empty((q.shape[0], 2 * q.shape[1]), dtype=np.float64)
    out[:, 0::2] = q & 15
    out[:, 1::2] = q >> 4
    return torch.from_numpy(out)


def pack(codes):
    """Bytes [N, K / 2] of codes [N, K] in 0 .. 15."""
    c = codes.to(torch.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def product_w4(x, q, scales, zeros):
    """(y, bound) of the 4-bit product."""
    t = x.dtype
    x, s = x.double().cpu(), scales.double().cpu()
    codes = unpack(q)
    N, K = codes.shape
    group = K // s.shape[1] if s.shape[1] else 1
    s = s.repeat_interleave(group, 1)
    z = torch.full_like(codes, 8.0) if zeros is None else zeros.double().cpu().repeat_interleave(group, 1)
    y = x @ ((codes - z) * s).T
    # codes enter as q + 128 (bfloat16) or q - 8 and the zero point takes the
    # offset out again: both sums count
    off = 128.0 if t == torch.bfloat16 else -8.0
    mag = x.abs() @ (((codes + off).abs() + (z + off).abs()) * s.abs()).T
    rel, absolute = half_step(t)
    return y, SUM * (K + 8) * mag + rel * y.abs() * (1 + SUM) + absolute


def assert_within(got, want, bound, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape, (got.shape, want.shape)
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d outside; first at %s: got %r, want %r, bound %r" % (
            what, int(bad.sum()), bad.numel(), i, float(got[i]), float(want[i]), float(bound[i])))
