"""Plain 64-bit forms of the operators around a training step's products, and
bounds on how far a correct kernel may be from them (test infrastructure).

A bound adds up, per element, what 32-bit arithmetic leaves (EPS: half a step,
2^-24, of each operation's result) and the rounding to the result's type (half
a step of it).
"""
from __future__ import annotations

import numpy as np
import torch

import _operators as plain

EPS = 2.0 ** -24
TYPES = plain.TYPES
half_step = plain.half_step
assert_within = plain.assert_within


def rounded(y, t):
    """Error of one rounding of 32-bit values near y to type t."""
    rel, absolute = half_step(t)
    return (rel * y.abs() + absolute) * (1 + 2 * rel) if t != torch.float32 else EPS * y.abs() + absolute


# ----------------------------------------------------------- layer_norm --

def norm_adds(cols):
    """Additions that one term of a row's sum goes through: a lane's share of
    the row (32 elements, or every 1024th chunk), six steps in a wave, sixteen
    waves."""
    return max(32, cols // 1024 + 8) + 24


def _norm_parts(x, eps):
    """(h, r, bound of h's error, relative bound of r's) for 64-bit x."""
    n = x.shape[1]
    k = norm_adds(n)
    mean = x.mean(1, keepdim=True)
    d = x - mean
    v = d.square().mean(1, keepdim=True)
    off = (k + 1) * EPS * x.abs().mean(1, keepdim=True)  # of the mean
    v_off = (k + 6) * EPS * v + off.square() + EPS * (v + eps)
    r = 1 / (v + eps).sqrt()
    r_rel = v_off / (v + eps) / 2 * 1.01 + 3 * EPS
    h = d * r
    return h, r, h.abs() * (r_rel + 2 * EPS) + r * off * (1 + r_rel), r_rel


def norm(x, weight, bias, eps=1e-5):
    """(y, bound)."""
    t = x.dtype
    x = x.double().cpu()
    w = torch.ones(x.shape[1], dtype=torch.float64) if weight is None else weight.double().cpu()
    b = torch.zeros(x.shape[1], dtype=torch.float64) if bias is None else bias.double().cpu()
    h, _, h_off, _ = _norm_parts(x, eps)
    y = h * w + b
    return y, h_off * w.abs() + 2 * EPS * y.abs() + rounded(y, t)


def norm_gradients(dy, x, weight, eps=1e-5, params=None):
    """((dx, dweight, dbias), their bounds)."""
    t, params = x.dtype, params or (x.dtype if weight is None else weight.dtype)
    x, dy = x.double().cpu(), dy.double().cpu()
    rows, n = x.shape
    k = norm_adds(n) + 2
    w = torch.ones(n, dtype=torch.float64) if weight is None else weight.double().cpu()
    h, r, h_off, r_rel = _norm_parts(x, eps)
    g = dy * w
    mg, mgh = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    mg_off = k * EPS * g.abs().mean(1, keepdim=True)
    mgh_off = k * EPS * (g * h).abs().mean(1, keepdim=True) + (g.abs() * h_off).mean(1, keepdim=True)
    dx = r * (g - mg - h * mgh)
    size = g.abs() + mg.abs() + (h * mgh).abs()
    dx_off = r * (mg_off + (h.abs() + h_off) * mgh_off + h_off * mgh.abs() + 4 * EPS * size) * (1 + r_rel) + r_rel * dx.abs()
    # sums over the rows: a lane's rows, up to 32 groups of lanes, up to 512
    # workgroups by sixteen waves; a lane has at most every 64th row
    adds = rows // 64 + 1 + 32 + 32 + 16 + 2
    dw, db = (dy * h).sum(0), dy.sum(0)
    dw_off = adds * EPS * (dy * h).abs().sum(0) + (dy.abs() * h_off).sum(0)
    db_off = adds * EPS * dy.abs().sum(0)
    return (dx, dw, db), (dx_off + rounded(dx, t), dw_off + rounded(dw, params), db_off + rounded(db, params))


# -------------------------------------------------------------- dropout --

def philox(counter, key):
    """Philox 4x32 with ten rounds of counters [n, 4] and one key of two words, as Python's whole numbers give it."""
    out = []
    for c in counter:
        c, (k0, k1) = [int(v) for v in c], [int(v) for v in key]
        for _ in range(10):
            a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
            c = [(b >> 32) ^ c[1] ^ k0, b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k1, a & 0xFFFFFFFF]
            k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
        out.append(c)
    return out


def kept(elements, p, seed, offset):
    """Whether dropout keeps elements number `elements` (an array of whole numbers)."""
    e = np.asarray(elements, dtype=np.uint64)
    block = e // np.uint64(8)
    m = np.uint64(0xFFFFFFFF)
    s = np.uint64(32)
    c = [block & m, block >> s, np.full_like(block, offset & 0xFFFFFFFF), np.full_like(block, offset >> 32)]
    for i in range(10):
        k0 = np.uint64(((seed & 0xFFFFFFFF) + i * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = np.uint64(((seed >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF)
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s) ^ c[1] ^ k0, b & m, (a >> s) ^ c[3] ^ k1, a & m]
    at = (e % np.uint64(8)).astype(np.int64)
    word = np.choose(at // 2, c)
    u = np.where(at % 2 == 1, word >> np.uint64(16), word & np.uint64(0xFFFF))
    return u.astype(np.int64) >= int(np.floor(p * 65536 + 0.5))


def dropout(x, p, seed, offset=0, residual=None):
    """(y, bound)."""
    t = x.dtype
    rows, cols = x.shape
    keep = torch.from_numpy(kept(np.arange(rows * cols), p, seed, offset)).reshape(rows, cols)
    d = int(np.floor(p * 65536 + 0.5))
    x = x.double().cpu()
    scaled = torch.where(keep, x * (65536 / (65536 - d) if d < 65536 else 0.0), torch.zeros((), dtype=torch.float64))
    y = scaled if residual is None else scaled + residual.double().cpu()
    return y, EPS * (scaled.abs() + y.abs()) + rounded(y, t)


# ------------------------------------------------- linear_cross_entropy --

def _wander(squares, n):
    """Error of 32-bit sums of n terms whose squares add up to `squares` (as in _tight)."""
    return (n / 32 + 24) * 2.0 ** -23 * 3 * squares.sqrt()


def loss(x, w, target, ignore=-100):
    """(loss, bound, parts) on x's device; parts are for loss_gradients.

    Of the sum of exponentials, all positive: each term is off by what its
    logarithm is, and every addition (34 in a wave, then one for each join,
    whose two exponentials count four) by EPS of the whole.
    """
    x, w = x.double(), w.double()
    T, D = x.shape
    V = w.shape[0]
    valid = target != ignore
    x = torch.where(valid[:, None], x, torch.zeros_like(x))  # (what a token that is ignored holds says nothing)
    l = x @ w.T
    l_off = _wander(x.square() @ w.square().T, D)
    top = l.max(1, keepdim=True).values
    e = (l - top).exp()
    s = e.sum(1, keepdim=True)
    p = e / s
    at = torch.where(valid, target, torch.zeros_like(target))[:, None]
    adds = 34 + 4 * (V // 4096 + 9)
    s_rel = (p * (l_off + (3 * (top - l) + 4) * EPS)).sum(1, keepdim=True) + adds * EPS + l_off.gather(1, l.argmax(1, keepdim=True))
    tl = l.gather(1, at)
    y = (top - tl + s.log())[:, 0]
    bound = (s_rel + l_off.gather(1, at) + 3 * EPS * (top - tl + s.log().abs() + 1))[:, 0] + 2 * EPS * y.abs()
    zero = torch.zeros_like(y)
    return torch.where(valid, y, zero), torch.where(valid, bound, zero), (x, w, valid, at, p, l, top, s, s_rel, l_off)


def loss_gradients(dloss, t, parts, rounded=True):
    """((dx, dw), their bounds); t: the operands' type; rounded: dl is rounded to
    it (as of more than 16 tokens)."""
    x, w, valid, at, p, l, top, s, s_rel, l_off = parts
    T, D = x.shape
    V = w.shape[0]
    rel, absolute = half_step(t)
    g = torch.where(valid, dloss.double(), torch.zeros_like(dloss.double()))[:, None]
    p_off = p * (l_off + s_rel + (5 * (top - l) + 5 * s.log().abs() + 80) * EPS)
    dl = p.clone()
    dl.scatter_add_(1, at, -torch.ones_like(s))
    p_off.scatter_add_(1, at, torch.full_like(s, 2 * EPS))
    small = 2.0 ** -40 if t == torch.float16 else absolute
    most = float(g.abs().max()) if T else 0.0
    rounding = rel * dl.abs() + small
    rounding.scatter_(1, at, torch.full_like(s, 4 * EPS))  # (what it takes there is put back)
    if not rounded:
        rounding = EPS * dl.abs()

    def sums(a, off, rnd, b, n, factor):
        y = a @ b
        walk = _wander((a.abs() + rnd).square() @ b.square(), n)
        bound = off @ b.abs() + 6 * (rnd.square() @ b.square()).sqrt() + walk
        y, bound = factor * y, factor.abs() * bound * (1 + 4 * EPS)
        return y, bound + rel * (1 + rel) * y.abs() + absolute

    one = torch.ones((), dtype=torch.float64, device=x.device)
    dx = sums(dl, p_off, rounding, w, V, g)
    gd = g * dl
    of_dw = rel * gd.abs() + most * small if rounded else EPS * gd.abs()
    dw = sums(gd.T, (g.abs() * p_off).T + 4 * EPS * gd.abs().T, of_dw.T, x, T, one)
    return (dx[0], dw[0]), (dx[1], dw[1])


def assert_near(got, want, bound, what=""):
    """assert_within on the device that the values are on."""
    bad = ~((got.double() - want).abs() <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d outside; first at %s: got %r, want %r, bound %r" % (
            what, int(bad.sum()), bad.numel(), i, float(got[i]), float(want[i]), float(bound[i])))
