"""Newton-Schulz on the host as the operator's documentation has it (test
infrastructure): the iteration in 64 bits with X, S and P rounded to binary16
times powers of two that bring the largest entry each can have near 2^14 (or
more, where that bound runs away), and P's rows times what rounding took from
its diagonal."""
from __future__ import annotations

import math

import torch

MUON = (3.4445, -4.7750, 2.0315)

# kernel and host round the same values but for one in five hundred that a
# 32-bit sum (off by 2^-20) takes the other way, from one half step to the other
SAME = 1.02


def held(g, steps=5, coefficients=MUON, eps=1e-7, corrected=True):
    """The result before its rounding to bfloat16; `corrected` false leaves P's diagonal as it is rounded."""
    x = g.double().cpu()
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    sigma = 1.0

    least = min(12, round(0.5 * math.log2(x.shape[1])))  # (where the bounds run away)

    def rounded(v, bound, least=0):
        k = 2.0 ** max(14 - math.ceil(math.log2(bound)), least)
        return (v * k).half().double() / k

    x = rounded(x / (x.norm() + eps), sigma, least)
    a, b, c = coefficients
    for k in range(steps):
        grid = torch.linspace(0, sigma, 4001, dtype=torch.float64)
        poly = a + b * grid ** 2 + c * grid ** 4
        s = rounded(x @ x.T, sigma ** 2)
        p = a * torch.eye(len(s), dtype=torch.float64) + b * s + c * (s @ s)
        p16 = rounded(p, float(poly.abs().max()))
        x = p16 @ x
        if corrected:
            d, d16 = p.diagonal(), p16.diagonal()
            x = x * torch.where(d16 == 0, torch.ones_like(d), d / d16)[:, None]
        sigma = float((poly * grid).abs().max())
        if k + 1 < steps:
            x = rounded(x, sigma, least)
    return x.T if tall else x


def distance(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


def entry_bound(exact, host):
    """How far an entry of a bfloat16 result may be from the exact one: its
    rounding, and eight times what the host's roundings of the iterates leave
    in its row or column on average (of some 10^7 errors spread like a normal
    distribution none is past six times that)."""
    e = (host - exact).square()
    spread = torch.maximum(e.mean(1, keepdim=True), e.mean(0, keepdim=True)).sqrt()
    return 2.0 ** -8 * exact.abs() + 8 * spread * (1 + 2.0 ** -8) + 2.0 ** -133


def noise(shape, t=torch.float32, seed=None):
    g = torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape) if seed is None else seed)) * 0.02
    return g.to(t)


def decaying(shape, tens, seed=0):
    """Singular values falling evenly in the logarithm from 1 to 10^-tens."""
    gen = torch.Generator().manual_seed(seed)
    m = min(shape)
    u, _ = torch.linalg.qr(torch.randn(shape[0], m, generator=gen, dtype=torch.float64))
    v, _ = torch.linalg.qr(torch.randn(shape[1], m, generator=gen, dtype=torch.float64))
    return (u @ torch.diag(torch.logspace(0, -tens, m, dtype=torch.float64)) @ v.T).float()


def with_small(shape, line, power):
    g = noise(shape)
    if line == "row":
        g[7] *= 10.0 ** power
    else:
        g[:, 7] *= 10.0 ** power
    return g


def own_rounding(exact):
    return distance(exact.bfloat16(), exact)
