"""ctypes bindings of the operators beside the product (argument marshalling only).

``libgated_nt.so``, ``liborthogonalize_ns.so`` and ``libgemv_w4.so`` with the
C ABIs of ``include/gated_nt.h``, ``include/orthogonalize_ns.h`` and
``include/gemv_w4.h``.  As in ``binding``, PyTorch supplies device memory
(results and workspaces) and the current stream, all arithmetic runs in the
libraries' HIP kernels, a missing library raises ``RuntimeError`` and a
refused call ``TypeError``, ``ValueError`` or ``GemmError``.  Nothing here
takes part in autograd: a training step calls the backward function itself.
A new result of inputs that require gradients raises when they are asked of it
(results in ``out`` and those of the training pair are the caller's affair).

Matrices may be views: the elements of a row are adjacent, rows may lie any
distance apart that does not make them overlap.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from .binding import GemmError, _stream

_HERE = os.path.dirname(os.path.abspath(__file__))

_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_p = ctypes.c_void_p
_int = ctypes.c_int

# library -> {function declared in include/<library>.h: its ctypes signature}
SIGNATURES = {
    "gated_nt": {
        "gated_nt": ([_p] * 5 + [_i64] * 7 + [_i32, _i32, _p, _i64, _p], _int),
        "gated_nt_backward": ([_p] * 8 + [_i64] * 10 + [_i32, _p, _i64, _p], _int),
        "gated_nt_saved_bytes": ([_i64] * 2, _i64),
        "gated_nt_workspace": ([_p] * 3 + [_i64] * 6, _i64),
        "gated_nt_backward_workspace": ([_i64] * 3, _i64),
        "gated_nt_version": ([], _int),
    },
    "orthogonalize_ns": {
        "orthogonalize_ns": ([_p, _p] + [_i64] * 7 + [_i32, _i32, ctypes.POINTER(ctypes.c_double), ctypes.c_double,
                                                      _p, _i64, _p], _int),
        "orthogonalize_ns_workspace": ([_i64] * 3, _i64),
        "orthogonalize_ns_version": ([], _int),
    },
    "gemv_w4": {
        "gemv_w4": ([_p] * 5 + [_i64] * 7 + [_i32, _p], _int),
        "gemv_w4_version": ([], _int),
    },
}

ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}
_TYPES = {torch.float16: 0, torch.bfloat16: 1}
_TYPES_AND_F32 = {**_TYPES, torch.float32: 2}

_libs = {}
_lock = threading.Lock()


def library_path(name: str) -> str:
    return os.path.join(_HERE, "lib%s.so" % name)


def load(name: str):
    """Load an operator's library once; raise if it has not been built."""
    lib = _libs.get(name)
    if lib is not None:
        return lib
    with _lock:
        if name not in _libs:
            path = library_path(name)
            if not os.path.exists(path):
                raise RuntimeError("lib%s.so is not built (%s); run "
                                   "`python -c 'import __graft_entry__ as g; g.build()'`" % (name, path))
            lib = ctypes.CDLL(path)
            for fn, (args, res) in SIGNATURES[name].items():
                f = getattr(lib, fn)
                f.argtypes = args
                f.restype = res
            _libs[name] = lib
    return _libs[name]


def _pitch(name, t, types, device=None, shape=None):
    """The row pitch of t, a GPU matrix of one of `types` whose rows do not overlap."""
    # (what holds is found out first and told apart only where it does not:
    # these checks are half of a short call's time on the host)
    if isinstance(t, torch.Tensor) and t.dtype in types and t.dim() == 2:
        index = t.get_device()
        rows, cols = size = t.shape
        ld, one = t.stride()
        if index >= 0 and (device is None or index == device) and (shape is None or size == shape) \
                and (one == 1 or cols <= 1) and (ld >= cols or rows <= 1):
            return ld if rows > 1 and cols > 0 else cols
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype not in types:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d).replace("torch.", "") for d in types),
                                                   str(t.dtype).replace("torch.", "")))
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError("%s must be a matrix%s, got %s" % (
            name, "" if shape is None else " of shape %s" % (tuple(shape),), tuple(t.shape)))
    if not t.is_cuda or (device is not None and t.get_device() != device):
        raise ValueError("%s must be on %s" % (name, "a GPU" if device is None else "the first operand's GPU"))
    raise ValueError("%s must have adjacent elements in a row and rows that do not overlap, got strides %s" % (
        name, t.stride()))


def _workspace(like, nbytes):
    """(tensor, address) of a workspace from torch's allocator: freed on
    return, and handed out again only to work later on the same stream."""
    if nbytes <= 0:
        return None, None
    w = like.new_empty(nbytes, dtype=torch.uint8)
    return w, w.data_ptr()


class _NoGradients(torch.autograd.Function):
    """The result of a call, of which no gradient can be had."""

    @staticmethod
    def forward(ctx, message, result, *inputs):
        ctx.message = message
        return result[0]  # (in a tuple: not an input itself)

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError(ctx.message)


def _without_gradients(result, message, *inputs):
    """`result` as it is, or one whose backward pass raises where autograd would have to go on to `inputs`."""
    if torch.is_grad_enabled() and any(t.requires_grad for t in inputs if t is not None):
        return _NoGradients.apply(message, (result,), *inputs)
    return result


def _call(library, name, device, *args):
    """Call an entry point on `device` and its current stream (the last argument)."""
    fn = getattr(load(library), name)
    if device == torch.cuda.current_device():
        rc = fn(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _stream(device))
    if rc != 0:
        raise GemmError(name, rc)


def _check_gated(x, w_gate, w_up):
    """(device, T, D, F, row pitches of x, w_gate and w_up)."""
    ldx = _pitch("x", x, _TYPES)
    device = x.get_device()
    types = (x.dtype,)
    ldg = _pitch("w_gate", w_gate, types, device)
    T, D = x.shape
    F, K = w_gate.shape
    if K != D:
        raise ValueError("need x [T, D] and w_gate, w_up [F, D], got %s and %s" % (tuple(x.shape), tuple(w_gate.shape)))
    ldu = _pitch("w_up", w_up, types, device, w_gate.shape)
    return device, T, D, F, ldx, ldg, ldu


def _gated(x, w_gate, w_up, activation, out, train):
    device, T, D, F, ldx, ldg, ldu = _check_gated(x, w_gate, w_up)
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError("activation must be one of %s, got %r" % (", ".join(sorted(ACTIVATIONS)), activation))
    if out is None:
        out = x.new_empty((T, F))
        ldh = F
    else:
        ldh = _pitch("out", out, (x.dtype,), device, (T, F))
    lib = load("gated_nt")
    saved = None
    if train:
        nbytes = lib.gated_nt_saved_bytes(T, F)
        if nbytes < 0:
            raise GemmError("gated_nt", 1)
        saved = x.new_empty(nbytes, dtype=torch.uint8)
    px, pg, pu = x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
    nbytes = lib.gated_nt_workspace(px, pg, pu, T, D, F, ldx, ldg, ldu)
    keep, workspace = _workspace(x, nbytes)
    _call("gated_nt", "gated_nt", device, px, pg, pu, out.data_ptr(), saved.data_ptr() if train else None, T, D, F, ldx,
          ldg, ldu, ldh, _TYPES[x.dtype], act, workspace, max(nbytes, 0))
    return out, saved


def gated_nt(x, w_gate, w_up, activation: str = "silu", out=None):
    """out[T, F] = act(x @ w_gate^T) * (x @ w_up^T) for x [T, D] and weights [F, D].

    float16 or bfloat16; ``activation`` is "silu" or "gelu_tanh".  Sums,
    activation and product in 32 bits, rounded once.  Enqueued on the current
    stream of x's device; returns ``out``.  Not differentiated by autograd:
    ``gated_nt_train`` and ``gated_nt_backward`` are its training form.
    """
    h = _gated(x, w_gate, w_up, activation, out, False)[0]
    if out is None and (x.requires_grad or w_gate.requires_grad or w_up.requires_grad):
        return _without_gradients(
            h, "gated_nt has no gradients in autograd: use gated_nt_train and gated_nt_backward", x, w_gate, w_up)
    return h


def gated_nt_train(x, w_gate, w_up, activation: str = "silu", out=None):
    """``gated_nt`` that also keeps what its backward pass reads: (out, saved).

    ``saved`` (8 bytes per output, 32-bit values in the library's own layout)
    is for ``gated_nt_backward`` with the same x and weights.  Neither requires
    gradients, whatever the inputs do.
    """
    return _gated(x, w_gate, w_up, activation, out, True)


def gated_nt_backward(dh, x, w_gate, w_up, saved, out=None):
    """The gradients (dx, dw_gate, dw_up) of ``gated_nt_train`` for the gradient dh [T, F] of its output.

    ``out``: three matrices to write them to, or None for new ones.  They are
    written, not added to.
    """
    device, T, D, F, ldx, ldg, ldu = _check_gated(x, w_gate, w_up)
    types = (x.dtype,)
    lddh = _pitch("dh", dh, types, device, (T, F))
    lib = load("gated_nt")
    need = lib.gated_nt_saved_bytes(T, F)
    nbytes = lib.gated_nt_backward_workspace(T, D, F)
    if need < 0 or nbytes < 0:
        raise GemmError("gated_nt_backward", 1)
    if not isinstance(saved, torch.Tensor) or saved.dtype != torch.uint8 or saved.dim() != 1 \
            or saved.numel() != need or not saved.is_contiguous() or (need and saved.get_device() != device):
        raise ValueError("saved must be what gated_nt_train returned for x, w_gate and w_up")
    if out is None:
        dx, dw_gate, dw_up = x.new_empty((T, D)), x.new_empty((F, D)), x.new_empty((F, D))
        lddx = lddg = lddu = D
    else:
        if len(out) != 3:
            raise ValueError("out must be the three matrices dx, dw_gate and dw_up")
        dx, dw_gate, dw_up = out
        lddx = _pitch("out's dx", dx, types, device, (T, D))
        lddg = _pitch("out's dw_gate", dw_gate, types, device, (F, D))
        lddu = _pitch("out's dw_up", dw_up, types, device, (F, D))
    keep, workspace = _workspace(x, nbytes)
    _call("gated_nt", "gated_nt_backward", device, dh.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
          saved.data_ptr(), dx.data_ptr(), dw_gate.data_ptr(), dw_up.data_ptr(), T, D, F, lddh, ldx, ldg, ldu, lddx, lddg,
          lddu, _TYPES[x.dtype], workspace, nbytes)
    return dx, dw_gate, dw_up


def orthogonalize_ns(g, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, out=None):
    """The update g [rows, cols] (or [batch, rows, cols]) with its singular values driven towards 1, in bfloat16.

    x = g / (|g|_F + eps), then ``steps`` times x = a x + (b s + c s s) x with
    s = x x^T.  ``coefficients`` is one triple (a, b, c), or one for each
    step.  g is float16, bfloat16 or float32; the iterates are held in
    binary16, hence the bfloat16 result, whose error for noise is up to 1.4
    times that of its rounding, and 5.6 times for singular values that fall off
    to 10^-4 (``include/orthogonalize_ns.h``).
    """
    if not isinstance(g, torch.Tensor):
        raise TypeError("g must be a torch tensor")
    if g.dim() not in (2, 3):
        raise ValueError("g must be [rows, cols] or [batch, rows, cols], got %s" % (tuple(g.shape),))
    steps = int(steps)
    if not 0 <= steps <= 64:
        raise ValueError("steps must be 0 .. 64, got %d" % steps)
    eps = float(eps)
    if not eps >= 0:
        raise ValueError("eps must not be negative, got %r" % eps)
    coefficients = coefficients.tolist() if hasattr(coefficients, "tolist") else list(coefficients)
    triples = [tuple(float(v) for v in c) for c in coefficients] if coefficients and hasattr(coefficients[0], "__len__") \
        else [tuple(float(v) for v in coefficients)] * steps
    if len(triples) != steps or any(len(c) != 3 for c in triples):
        raise ValueError("coefficients must be one triple, or one for each of the %d steps" % steps)
    batch = g.shape[0] if g.dim() == 3 else 1
    rows, cols = g.shape[-2:]

    def first(t):  # one matrix of the batch (of an empty one: none of its rows)
        return t if t.dim() == 2 else t[0] if t.shape[0] else t.new_empty(0, cols)

    ldg = _pitch("g", first(g), _TYPES_AND_F32)
    device = g.get_device()
    new = out is None
    if new:
        out = g.new_empty(g.shape, dtype=torch.bfloat16)
    if not isinstance(out, torch.Tensor) or out.shape != g.shape:
        raise ValueError("out must be a bfloat16 tensor of g's shape %s" % (tuple(g.shape),))
    ldo = _pitch("out", first(out), (torch.bfloat16,), device)
    if g.numel() == 0:
        return out
    stride_g, stride_o = (t.stride(0) if t.dim() == 3 and batch > 1 else 0 for t in (g, out))
    if batch > 1 and (stride_g < 0 or stride_o < (rows - 1) * ldo + cols):
        raise ValueError("out's matrices must lie one after another and not overlap, got strides %s" % (out.stride(),))
    lib = load("orthogonalize_ns")
    nbytes = lib.orthogonalize_ns_workspace(batch, rows, cols)
    if nbytes < 0:
        raise GemmError("orthogonalize_ns", 1)
    keep, workspace = _workspace(g, nbytes)
    flat = (ctypes.c_double * max(1, 3 * steps))(*(v for c in triples for v in c))
    _call("orthogonalize_ns", "orthogonalize_ns", device, g.data_ptr(), out.data_ptr(), batch, rows, cols, ldg, stride_g,
          ldo, stride_o, _TYPES_AND_F32[g.dtype], steps, flat, eps, workspace, nbytes)
    if new and g.requires_grad:
        return _without_gradients(out, "orthogonalize_ns has no gradients in autograd", g)
    return out


def gemv_w4(x, q, scales, zeros=None, out=None):
    """out[M, N] = x[M, K] @ w^T for 4-bit weights w[n, k] = (q[n, k] - zeros[n, k // group]) * scales[n, k // group].

    ``q`` is uint8 [N, K / 2], even k in the low half of a byte; ``scales``
    [N, K / group] of x's type gives the group (a power of two from 32 on, or
    K); ``zeros`` likewise, or None for 8.  x is float16 or bfloat16.
    Enqueued on the current stream of x's device; returns ``out``.
    """
    ldx = _pitch("x", x, _TYPES)
    device = x.get_device()
    types = (x.dtype,)
    ldq = _pitch("q", q, (torch.uint8,), device)
    M, K = x.shape
    N, half = q.shape
    if K % 32 or half * 2 != K:
        raise ValueError("need x [M, K] and q [N, K / 2] with K a multiple of 32, got %s and %s" % (
            tuple(x.shape), tuple(q.shape)))
    pq = q.data_ptr()
    if (pq % 16 or (N > 1 and ldq % 16)) and N and K:
        raise ValueError("q's rows must start on 16 bytes")
    _pitch("scales", scales, types, device)
    rows, groups = scales.shape
    if rows != N or not scales.is_contiguous():
        raise ValueError("scales must be contiguous [%d, groups], got %s" % (N, tuple(scales.shape)))
    if zeros is not None:
        _pitch("zeros", zeros, types, device, scales.shape)
        if not zeros.is_contiguous():
            raise ValueError("zeros must be contiguous")
    group = K // groups if groups and K % groups == 0 else 0
    if K and (group == 0 or ((group < 32 or group & (group - 1)) and group != K)):
        raise ValueError("K / scales.shape[1] must be a power of two from 32 on, or K: got %d / %d" % (K, groups))
    new = out is None
    if new:
        out = x.new_empty((M, N))
        ldy = N
    else:
        ldy = _pitch("out", out, types, device, (M, N))
    _call("gemv_w4", "gemv_w4", device, x.data_ptr(), pq, scales.data_ptr(), None if zeros is None else zeros.data_ptr(),
          out.data_ptr(), M, N, K, group, ldx, ldq if N > 1 else half, ldy, _TYPES[x.dtype])
    if new and (x.requires_grad or scales.requires_grad or (zeros is not None and zeros.requires_grad)):
        return _without_gradients(out, "gemv_w4 has no gradients in autograd", x, scales, zeros)
    return out
