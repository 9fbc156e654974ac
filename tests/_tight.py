"""Bounds near what the operators' roundings leave (test infrastructure).

Where ``_operators`` allows each of a sum's additions a step of the sum of all
magnitudes, which at long sums is more than the result, these follow how the
sums come about:
* a sum of n terms of either sign wanders as far as the root of their squares'
  sum, R, and seldom past three times that; the matrix cores add 32 terms at
  once, waves and parts a few dozen results more: n / 32 + 24 additions, each
  off by a step (2^-23) of what it adds to;
* operands rounded to the type are each off by half a step at most, either way:
  what reaches a sum of them is spread by their root of squares over sqrt 3, and
  six half steps of that root are ten times the spread.
The tests on the host show what the bounds reject: zeros, and results that lack
a piece of the sum.
"""
from __future__ import annotations

import torch

import _operators as plain

FUN = plain.FUN


def wander(squares, n):
    """Error of 32-bit sums of n terms whose squares add up to `squares`."""
    return (n / 32 + 24) * 2.0 ** -23 * 3 * squares.sqrt()


def products(x, w):
    return x @ w.T, wander(x.square() @ w.square().T, x.shape[1])


def gated(x, wg, wu, act):
    rel, absolute = plain.half_step(x.dtype)
    x, wg, wu = (v.double().cpu() for v in (x, wg, wu))
    (g, eg), (u, eu) = products(x, wg), products(x, wu)
    a, _ = plain.activation(g, act)
    h = a * u
    return h, 1.13 * u.abs() * eg + a.abs() * eu + 1.13 * eg * eu + (FUN + rel * (1 + FUN)) * h.abs() + absolute


def gradients(dh, x, wg, wu, act):
    rel, absolute = plain.half_step(x.dtype)
    dh, x, wg, wu = (v.double().cpu() for v in (dh, x, wg, wu))
    T, F = dh.shape
    (g, eg), (u, eu) = products(x, wg), products(x, wu)
    a, da = plain.activation(g, act)
    dg, du = dh * u * da, dh * a
    # what 32-bit values are off by, and the rounding to the type (binary16:
    # steps of 2^-24 after dh's largest entry is brought to 2^-4 or more)
    step = absolute if rel != 2.0 ** -11 else float(dh.abs().max()) * 2.0 ** -20
    g_off = dh.abs() * (0.8 * u.abs() * eg + 1.13 * eu + 0.8 * eg * eu + FUN * (1 + g.abs()) * u.abs())
    u_off = dh.abs() * (1.13 * eg + FUN * a.abs())
    g_round, u_round = rel * dg.abs() + step, rel * du.abs() + step

    def sums(parts, n):
        """(sum of a @ b over the parts, its bound)"""
        y = sum(d @ b for d, _, _, b in parts)
        off = sum(o @ b.abs() for _, o, _, b in parts)
        spread = sum(r.square() @ b.square() for _, _, r, b in parts).sqrt()
        walk = wander(sum((d.abs() + r).square() @ b.square() for d, _, r, b in parts), n)
        return y, off + 6 * spread + walk + rel * (1 + rel) * y.abs() + absolute

    dx = sums([(dg, g_off, g_round, wg), (du, u_off, u_round, wu)], 2 * F)
    dwg = sums([(dg.T, g_off.T, g_round.T, x)], T)
    dwu = sums([(du.T, u_off.T, u_round.T, x)], T)
    return [v[0] for v in (dx, dwg, dwu)], [v[1] for v in (dx, dwg, dwu)]


def product_w4(x, q, scales, zeros):
    t = x.dtype
    rel, absolute = plain.half_step(t)
    x, s = x.double().cpu(), scales.double().cpu()
    codes = plain.unpack(q)
    K = codes.shape[1]
    group = K // s.shape[1]
    s = s.repeat_interleave(group, 1)
    z = torch.full_like(codes, 8.0) if zeros is None else zeros.double().cpu().repeat_interleave(group, 1)
    y = x @ ((codes - z) * s).T
    off = 128.0 if t == torch.bfloat16 else -8.0
    terms = x.square() @ (((codes + off).abs() + (z + off).abs()) * s).square().T
    return y, wander(terms, K) + rel * (1 + 2.0 ** -20) * y.abs() + absolute


def rms(v):
    return float(v.double().square().mean().sqrt())


def near(got, want, bound, times, t):
    """Whether every entry is within its bound and, of enough of them (and with
    `times` given), the root mean square of the errors within `times` that of
    rounding the exact values."""
    got = got.double().cpu()
    if not ((got - want).abs() <= bound).all():
        return False
    return times is None or want.numel() < 256 or rms(got - want) <= times * rms(want.to(t).double() - want)


# of results: their own rounding and next to nothing; of the gated layer's
# gradients: as much again from dG and dU, sqrt 2 of one (and a tenth)
RESULT = 1.1


def gradient_times(T, F):
    """The latter is an average over the T F roundings of dG, weighted by their
    squares.  Those, products of three about normal factors, have a kurtosis of
    27, so that of N of them the average is spread by sqrt(27 * 1.8 / N): 0.07
    of itself for 10^4, of which 1.56^2 - 2 = 0.43 is six, but 0.8 for 66.  With
    fewer there is no average to speak of, only the bound of each entry."""
    return 1.56 if T * F >= 10 ** 4 else None
