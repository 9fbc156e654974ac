"""ctypes bindings of the operators around a training step's products (argument
marshalling only): the layer norm, dropout with the sum of a residual, and the
loss over a vocabulary, each with its backward pass.

``liblayer_norm.so``, ``libdropout.so`` and ``liblinear_cross_entropy.so`` with
the C ABIs of ``include/layer_norm.h``, ``include/dropout.h`` and
``include/linear_cross_entropy.h``.  As in ``operators``: PyTorch supplies device
memory and the current stream, a missing library raises ``RuntimeError`` and a
refused call ``TypeError``, ``ValueError`` or ``GemmError``, matrices may be
views whose rows' elements are adjacent, and nothing takes part in autograd: a
training step calls the backward functions itself.  A new result raises when
gradients are asked of it that it has none for: those of the inputs of
``layer_norm``, ``dropout`` and ``linear_cross_entropy``, and those of a backward
function's dy or dloss (a second derivative).  An operand with a tangent of
forward-mode differentiation is refused.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from .binding import GemmError
from .operators import _TYPES, _TYPES_AND_F32, _call, _pitch, _refuse_tangent, _without_gradients, _workspace, load

_WORDS = 1 << 64


def _new(x, pitch):
    """A new matrix like x, whose rows are `pitch` apart, with rows that are adjacent."""
    return torch.empty_like(x, requires_grad=False) if pitch == x.shape[1] and x.is_contiguous() else x.new_empty(x.shape)


def _vector(name, t, types, device, size):
    """Check t, `size` adjacent elements of one of `types` on `device`."""
    if forward_ad._current_level >= 0:
        _refuse_tangent(name, t)
    # (what holds is found out first and told apart only where it does not)
    if isinstance(t, torch.Tensor) and t.dtype in types and t.shape == (size,) and t.get_device() == device and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype not in types:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d).replace("torch.", "") for d in types),
                                                   str(t.dtype).replace("torch.", "")))
    if t.dim() != 1 or t.shape[0] != size or not t.is_contiguous():
        raise ValueError("%s must be contiguous [%d], got %s" % (name, size, tuple(t.shape)))
    if t.get_device() != device:
        raise ValueError("%s must be on the first operand's GPU" % name)


# ----------------------------------------------------------- layer_norm --

def _check_norm(x, weight, bias):
    """(device, pitch of x, type of the parameters)."""
    ldx = _pitch("x", x, _TYPES_AND_F32)
    device = x.get_device()
    types = (x.dtype, torch.float32)
    if weight is not None:
        _vector("weight", weight, types, device, x.shape[1])
        types = (weight.dtype,)  # one type for both
    if bias is not None:
        _vector("bias", bias, types, device, x.shape[1])
        types = (bias.dtype,)
    return device, ldx, types[0]


def _norm(x, weight, bias, eps, out, train):
    device, ldx, params = _check_norm(x, weight, bias)
    eps = float(eps)
    if not eps >= 0:
        raise ValueError("eps must not be negative, got %r" % eps)
    rows, cols = x.shape
    if out is None:
        out = _new(x, ldx)
        ldy = cols
    else:
        ldy = _pitch("out", out, (x.dtype,), device, (rows, cols))
    saved = x.new_empty((rows, 2), dtype=torch.float32) if train else None
    _call("layer_norm", "layer_norm", device, x.data_ptr(), None if weight is None else weight.data_ptr(),
          None if bias is None else bias.data_ptr(), out.data_ptr(), saved.data_ptr() if train else None, rows, cols, ldx, ldy,
          _TYPES_AND_F32[x.dtype], _TYPES_AND_F32[params], eps)
    return out, saved


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None):
    """(x - mean) / sqrt(variance + eps) * weight + bias over the rows of x [rows, cols].

    float16, bfloat16 or float32; weight and bias [cols], both of x's type or
    both float32, or None for 1 and 0.  Statistics in 32 bits, rounded once.
    Enqueued on the current stream of x's device; returns ``out``.  Not
    differentiated by autograd: ``layer_norm_train`` and
    ``layer_norm_backward`` are its training form.
    """
    y = _norm(x, weight, bias, eps, out, False)[0]
    if out is None and (x.requires_grad or (weight is not None and weight.requires_grad) or (bias is not None and bias.requires_grad)):
        return _without_gradients(
            y, "layer_norm has no gradients in autograd: use layer_norm_train and layer_norm_backward", x, weight, bias)
    return y


def layer_norm_train(x, weight=None, bias=None, eps: float = 1e-5, out=None):
    """``layer_norm`` that also keeps what its backward pass reads: (out, saved).

    ``saved`` is float32 [rows, 2]: each row's mean and 1 / sqrt(variance + eps).
    Neither requires gradients, whatever the inputs do.
    """
    return _norm(x, weight, bias, eps, out, True)


def layer_norm_backward(dy, x, weight, bias, saved, out=None):
    """The gradients (dx, dweight, dbias) of ``layer_norm_train`` for the gradient dy of its output.

    None for a weight or bias that is None.  ``out``: the three to write them
    to (None where there is none), or None for new ones.  They are written,
    not added to.
    """
    device, ldx, params = _check_norm(x, weight, bias)
    rows, cols = x.shape
    lddy = _pitch("dy", dy, (x.dtype,), device, (rows, cols))
    if not isinstance(saved, torch.Tensor) or saved.dtype != torch.float32 or tuple(saved.shape) != (rows, 2) \
            or not saved.is_contiguous() or saved.get_device() != device:
        raise ValueError("saved must be what layer_norm_train returned for x")
    if out is None:
        dx = _new(x, ldx)
        dw, db = (None if t is None else torch.empty_like(t, requires_grad=False) for t in (weight, bias))
        lddx = cols
    else:
        if len(out) != 3:
            raise ValueError("out must be dx, dweight and dbias")
        dx, dw, db = out
        lddx = _pitch("out's dx", dx, (x.dtype,), device, (rows, cols))
        for name, t, of in (("dweight", dw, weight), ("dbias", db, bias)):
            if (t is None) != (of is None):
                raise ValueError("out's %s must be given where its parameter is, and only there" % name)
            if t is not None:
                _vector("out's " + name, t, (params,), device, cols)
    nbytes = load("layer_norm").layer_norm_backward_workspace(rows, cols)
    if nbytes < 0:
        raise GemmError("layer_norm_backward", 1)
    keep, workspace = _workspace(x, nbytes)
    _call("layer_norm", "layer_norm_backward", device, dy.data_ptr(), x.data_ptr(), None if weight is None else weight.data_ptr(),
          saved.data_ptr(), dx.data_ptr(), None if dw is None else dw.data_ptr(), None if db is None else db.data_ptr(), rows, cols,
          lddy, ldx, lddx, _TYPES_AND_F32[x.dtype], _TYPES_AND_F32[params], workspace, nbytes)
    if out is None and dy.requires_grad:
        return tuple(None if t is None else _without_gradients(t, "layer_norm_backward has no gradients in autograd", dy)
                     for t in (dx, dw, db))
    return dx, dw, db


# -------------------------------------------------------------- dropout --

def _dropout(x, p, seed, offset, residual, out):
    ldx = _pitch("x", x, _TYPES_AND_F32)
    device = x.get_device()
    p = float(p)
    if not 0 <= p <= 1:
        raise ValueError("p must be 0 .. 1, got %r" % p)
    state = None
    if isinstance(seed, torch.Tensor):
        _vector("seed, if not a number,", seed, (torch.int64,), device, 2)
        state, seed = seed.data_ptr(), 0
    seed, offset = int(seed), int(offset)
    if not 0 <= seed < _WORDS or not 0 <= offset < _WORDS:
        raise ValueError("seed and offset must be 0 .. 2^64 - 1, got %d and %d" % (seed, offset))
    ldr = 0
    if residual is not None:
        ldr = _pitch("residual", residual, (x.dtype,), device, x.shape)
    if out is None:
        out = _new(x, ldx)
        ldy = x.shape[1]
    else:
        ldy = _pitch("out", out, (x.dtype,), device, x.shape)
    _call("dropout", "dropout", device, x.data_ptr(), None if residual is None else residual.data_ptr(), out.data_ptr(), *x.shape,
          ldx, ldr, ldy, _TYPES_AND_F32[x.dtype], p, seed, offset, state)
    return out


def dropout(x, p: float, seed, offset: int = 0, residual=None, out=None):
    """x [rows, cols] with each element dropped with probability p and the others scaled by 1 / (1 - p), plus residual.

    The mask is drawn from ``seed`` and ``offset`` by a counter-based generator
    (``include/dropout.h``) and not stored: the same numbers give the same mask,
    another offset an independent one.  p is held to 2^-17.  ``seed`` may be an
    int64 tensor (seed, offset) on x's GPU, read when the call runs, to whose
    offset ``offset`` is added: a captured graph then draws anew each time it is
    replayed.  float16, bfloat16 or float32; ``out`` may be x or residual.  Not
    differentiated by autograd: ``dropout_backward`` gives x's gradient, and the
    residual's is the result's own.
    """
    y = _dropout(x, p, seed, offset, residual, out)
    if out is None and (x.requires_grad or (residual is not None and residual.requires_grad)):
        return _without_gradients(y, "dropout has no gradients in autograd: use dropout_backward", x, residual)
    return y


def dropout_backward(dy, p: float, seed, offset: int = 0, out=None):
    """x's gradient for the gradient dy of ``dropout``'s result with the same p, seed and offset; ``out`` may be dy."""
    dx = _dropout(dy, p, seed, offset, None, out)
    if out is None and dy.requires_grad:
        return _without_gradients(dx, "dropout_backward has no gradients in autograd", dy)
    return dx


# ------------------------------------------------- linear_cross_entropy --

def _strided(name, t, dtype, device, size):
    """The stride of t, `size` elements of `dtype` on `device`, any distance apart."""
    if forward_ad._current_level >= 0:
        _refuse_tangent(name, t)
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, str(dtype).replace("torch.", ""), str(t.dtype).replace("torch.", "")))
    if t.dim() != 1 or t.shape[0] != size:
        raise ValueError("%s must be [%d], got %s" % (name, size, tuple(t.shape)))
    if t.get_device() != device:
        raise ValueError("%s must be on the first operand's GPU" % name)
    return t.stride(0) if size > 1 else 1


def _check_loss(x, w, target):
    """(device, T, D, V, pitches of x and w, stride of target)."""
    ldx = _pitch("x", x, _TYPES)
    device = x.get_device()
    ldw = _pitch("w", w, (x.dtype,), device)
    T, D = x.shape
    V, K = w.shape
    if K != D or V == 0:
        raise ValueError("need x [T, D] and w [V, D] with V above 0, got %s and %s" % (tuple(x.shape), tuple(w.shape)))
    return device, T, D, V, ldx, ldw, _strided("target", target, torch.int64, device, T)


def _ignored(index):
    index = int(index)
    if not -_WORDS // 2 <= index < _WORDS // 2:
        raise ValueError("ignore_index must fit 64 bits, got %d" % index)
    return index


def _loss(x, w, target, ignore_index, out, train):
    device, T, D, V, ldx, ldw, stride = _check_loss(x, w, target)
    ignored = _ignored(ignore_index)
    if out is None:
        out = x.new_empty(T, dtype=torch.float32)
    else:
        _vector("out", out, (torch.float32,), device, T)
    saved = x.new_empty((T, 3), dtype=torch.float32) if train else None
    px, pw = x.data_ptr(), w.data_ptr()
    nbytes = load("linear_cross_entropy").linear_cross_entropy_workspace(px, pw, T, D, V, ldx, ldw)
    if nbytes < 0:
        raise GemmError("linear_cross_entropy", 1)
    keep, workspace = _workspace(x, nbytes)
    _call("linear_cross_entropy", "linear_cross_entropy", device, px, pw, target.data_ptr(), out.data_ptr(),
          saved.data_ptr() if train else None, T, D, V, ldx, ldw, stride, _TYPES[x.dtype], ignored, workspace, nbytes)
    return out, saved


def linear_cross_entropy(x, w, target, ignore_index: int = -100, out=None):
    """loss[t] = log sum_v exp(l[t, v]) - l[t, target[t]] of l = x @ w^T, for x [T, D], w [V, D] and int64 target [T].

    float16 or bfloat16; losses float32, one for each token, 0 where target is
    ``ignore_index`` (whatever x holds there), NaN where it is neither that nor
    in 0 .. V - 1.  l is summed in 32 bits and not kept.  Enqueued on the
    current stream of x's device; returns ``out``.  Not differentiated by
    autograd: ``linear_cross_entropy_train`` and
    ``linear_cross_entropy_backward`` are its training form.
    """
    loss = _loss(x, w, target, ignore_index, out, False)[0]
    if out is None and (x.requires_grad or w.requires_grad):
        return _without_gradients(loss, "linear_cross_entropy has no gradients in autograd: use linear_cross_entropy_train and "
                                  "linear_cross_entropy_backward", x, w)
    return loss


def linear_cross_entropy_train(x, w, target, ignore_index: int = -100, out=None):
    """``linear_cross_entropy`` that also keeps what its backward pass reads: (out, saved).

    ``saved`` is float32 [T, 3]: each row's largest l, the sum of exp(l -
    largest), and the target's l.  Neither requires gradients, whatever the
    inputs do.
    """
    return _loss(x, w, target, ignore_index, out, True)


def linear_cross_entropy_backward(dloss, x, w, target, saved, ignore_index: int = -100, out=None):
    """The gradients (dx, dw) of ``linear_cross_entropy_train`` for the gradient dloss [T] (float32) of its losses.

    dloss may be one number expanded.  ``out``: two matrices to write them to,
    or None for new ones.  They are written, not added to.
    """
    device, T, D, V, ldx, ldw, stride = _check_loss(x, w, target)
    types = (x.dtype,)
    ignored = _ignored(ignore_index)
    sg = _strided("dloss", dloss, torch.float32, device, T)
    if not isinstance(saved, torch.Tensor) or saved.dtype != torch.float32 or tuple(saved.shape) != (T, 3) \
            or not saved.is_contiguous() or saved.get_device() != device:
        raise ValueError("saved must be what linear_cross_entropy_train returned for x, w and target")
    if out is None:
        dx, dw = x.new_empty((T, D)), x.new_empty((V, D))
        lddx = lddw = D
    else:
        if len(out) != 2:
            raise ValueError("out must be the two matrices dx and dw")
        dx, dw = out
        lddx = _pitch("out's dx", dx, types, device, (T, D))
        lddw = _pitch("out's dw", dw, types, device, (V, D))
    px, pw = x.data_ptr(), w.data_ptr()
    nbytes = load("linear_cross_entropy").linear_cross_entropy_backward_workspace(px, pw, T, D, V, ldx, ldw)
    if nbytes < 0:
        raise GemmError("linear_cross_entropy_backward", 1)
    keep, workspace = _workspace(x, nbytes)
    _call("linear_cross_entropy", "linear_cross_entropy_backward", device, dloss.data_ptr(), px, pw, target.data_ptr(),
          saved.data_ptr(), dx.data_ptr(), dw.data_ptr(), T, D, V, sg, ldx, ldw, stride, lddx, lddw, _TYPES[x.dtype],
          ignored, workspace, nbytes)
    if out is None and dloss.requires_grad:
        return tuple(_without_gradients(t, "linear_cross_entropy_backward has no gradients in autograd", dloss) for t in (dx, dw))
    return dx, dw
