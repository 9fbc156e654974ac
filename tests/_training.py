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
