"""The memory-bound layers of a pre-norm training step (include/gclip_layer.h):
layer norm, dropout from a counter-based generator, and the residual step
that runs both in one pass, forward and backward.

As in the rest of the package the functions named like the C ABI take its
structures with raw device addresses, and the others torch tensors, which
serve as device memory and streams: every step runs in the HIP kernels.

- ``layer_norm_forward`` / ``_backward``, ``dropout_forward`` / ``_backward``
  and ``residual_norm_forward`` / ``_backward`` are the passes themselves, for
  a program that writes its own backward pass: the weights' gradients go into
  buffers of the caller's, added to what the microbatches before left there
  when ``accumulate`` is set, from where a ``GradList`` clips them.
- ``layer_norm``, ``dropout`` and ``residual_norm`` are the same under
  autograd, in its backward mode: tensors with a tangent are refused, and so
  is tracing.  To capture a training step into a graph, capture the passes; a
  captured autograd backward needs leaves that no eager graph holds.

A matrix is a tensor whose last dimension is adjacent in memory and whose
other dimensions lie at one distance (a contiguous tensor, a slice of the
columns of a wider one, one row expanded).
"""
import ctypes

try:
    import torch
except ImportError:  # the functions named like the C ABI do without it
    torch = None

from . import _check, _lib
from ._lib import GCLIP_BF16, GCLIP_F16, GCLIP_F32, GclipDropout, GclipLayerBackward, GclipLayerForward

_byref = ctypes.byref


# ---------------------------------------------------------------- C ABI names
def gclip_layernorm_forward(args, stream):
    _check(_lib.lib.gclip_layernorm_forward(_byref(args), stream), "gclip_layernorm_forward")


def gclip_layernorm_backward(args, stream):
    _check(_lib.lib.gclip_layernorm_backward(_byref(args), stream), "gclip_layernorm_backward")


def gclip_residual_forward(args, drop, stream):
    _check(_lib.lib.gclip_residual_forward(_byref(args), _byref(drop) if drop is not None else None, stream),
           "gclip_residual_forward")


def gclip_residual_backward(args, drop, stream):
    _check(_lib.lib.gclip_residual_backward(_byref(args), _byref(drop) if drop is not None else None, stream),
           "gclip_residual_backward")


def gclip_dropout_apply(x, ldx, y, ldy, rows, size, dtype, drop, stream):
    _check(_lib.lib.gclip_dropout_apply(x, ldx, y, ldy, rows, size, dtype, _byref(drop), stream),
           "gclip_dropout_apply")


def gclip_layer_workspace(rows, size):
    return _lib.lib.gclip_layer_workspace(rows, size)


# ---------------------------------------------------------------- tensors as operands
if torch is not None:
    _CODES = {torch.float32: GCLIP_F32, torch.float16: GCLIP_F16, torch.bfloat16: GCLIP_BF16}
    _F32 = torch.float32
    _increment_version = torch.autograd.graph.increment_version
    # a small call takes a few microseconds: torch.cuda.current_stream() alone
    # would be a third of it
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)


def _counted(mask, device):
    """The mask's structure; its counter has to be on the device that reads it,
    and where it was when the mask was made."""
    counter = mask.counter
    if counter is not None:
        if counter.get_device() != device:
            raise ValueError(f"the mask's counter is on {counter.device}")
        if counter.data_ptr() != mask.args.d_step or counter.numel() < 1:
            raise ValueError("the mask's counter has another storage than when the mask was made")
    return mask.args


def _matrix(x, name):
    """(device index, rows, size, ld, dtype code) of the matrix that a call
    goes by; its device has to be the current one: kernels are enqueued
    there."""
    if torch._C._is_tracing():
        raise RuntimeError("the layers cannot be traced: a trace records none of their kernels")
    code = _CODES.get(x.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {x.dtype}")
    device = x.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a device tensor")
    if device != _current_device():
        raise ValueError(f"{name} is on device {device}, the current one is {_current_device()}")
    shape = x.shape
    if not shape:
        raise ValueError(f"{name} must have at least one dimension")
    size = shape[-1]
    if size:
        return device, x.numel() // size, size, size if x.is_contiguous() else _ld(x, name), code
    rows = 1
    for n in shape[:-1]:
        rows *= n
    return device, rows, 0, 0, code


def _ld(t, name):
    """Distance of a matrix's rows in elements."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2 and stride[1] == 1 and shape[0] > 1:
        return stride[0]
    if t.is_contiguous() or t.numel() == 0:
        return shape[-1]
    lead = [(n, s) for n, s in zip(shape[:-1], stride[:-1]) if n != 1]
    if (shape[-1] != 1 and stride[-1] != 1) or any(a[1] != b[0] * b[1] for a, b in zip(lead, lead[1:])):
        raise ValueError(f"{name}: the last dimension must be adjacent in memory and the others at one distance; "
                         f"a contiguous() copy is")
    return lead[-1][1] if lead else shape[-1]


def _like(t, x, name):
    """ld of a matrix of x's shape, dtype and device."""
    if t.dtype != x.dtype:
        raise TypeError(f"{name} must have dtype {x.dtype}, not {t.dtype}")
    if t.shape != x.shape or t.get_device() != x.get_device():
        raise ValueError(f"{name} must have shape {tuple(x.shape)} on {x.device}")
    return t.shape[-1] if t.is_contiguous() else _ld(t, name)


def _vector(t, n, x, name):
    """Address of a contiguous binary32 vector, or one of x's dtype."""
    if t.dtype != _F32 and t.dtype != x.dtype:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.numel() != n or not t.is_contiguous() or t.get_device() != x.get_device():
        raise ValueError(f"{name} must hold {n} contiguous elements on {x.device}")
    return t.data_ptr()


def _statistic(t, n, x, name):
    if t.dtype != _F32:
        raise TypeError(f"{name} must be float32, not {t.dtype}")
    return _vector(t, n, x, name)


def _there(stream, f, *args):
    """f(*args) on another stream than the current one: its new tensors are
    that stream's, and its operands' memory is not given out before it has
    run."""
    for t in args:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
        elif isinstance(t, DropoutMask) and t.counter is not None:
            t.counter.record_stream(stream)
    with torch.cuda.stream(stream):
        return f(*args)


def _wrote(*tensors):
    """Autograd may have saved what a caller gives to be written: as after an
    in-place operation of torch, its backward pass then refuses it."""
    for t in tensors:
        if t is not None:
            _increment_version(t)


# ---------------------------------------------------------------- dropout
class DropoutMask:
    """Which elements a dropout keeps, as a function of its arguments alone:
    nothing is stored, and the backward pass takes the same object.

    p        probability of dropping, to 16 bits (0 <= p <= 1)
    seed     64 bits
    step     32 bits: another mask every step ...
    site     32 bits: ... and for every place of a step that drops
    counter  optional device tensor whose first int32 is added to step: a
             captured graph takes it anew at each replay (``counter.add_(1)``
             between the replays, and not between a pass and its backward)

    A mask does not change: ``at`` gives another one.
    """

    __slots__ = ("p", "seed", "step", "site", "counter", "args")

    def __init__(self, p, seed, step=0, site=0, counter=None):
        p = float(p)
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p must be in [0, 1], not {p}")
        if not (0 <= seed < 1 << 64 and 0 <= step < 1 << 32 and 0 <= site < 1 << 32):
            raise ValueError("seed takes 64 bits, step and site take 32")
        address = None
        if counter is not None:
            if counter.dtype != torch.int32 or not counter.is_cuda or counter.numel() < 1:
                raise ValueError("counter must be an int32 device tensor")
            address = counter.data_ptr()
        values = p, seed, step, site, counter, GclipDropout(p, seed, step, site, address)
        for name, value in zip(self.__slots__, values):
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        raise AttributeError("a mask does not change; at() gives another one")

    def __reduce__(self):
        return DropoutMask, (self.p, self.seed, self.step, self.site, self.counter)

    def at(self, step=None, site=None):
        """The mask of another step or site."""
        return DropoutMask(self.p, self.seed, self.step if step is None else step,
                           self.site if site is None else site, self.counter)

    @property
    def drops(self):
        """Whether p is large enough to drop anything."""
        return self.p >= 2.0 ** -17


def dropout_forward(x, mask, out=None, stream=None):
    """x where the mask keeps it, times 1 / (1 - p); else 0.  out may be x."""
    if stream is not None:
        return _there(stream, dropout_forward, x, mask, out)
    given = out
    device, rows, size, ld, code = _matrix(x, "x")
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        ldo = size
    else:
        ldo = _like(out, x, "out")
    gclip_dropout_apply(x.data_ptr(), ld, out.data_ptr(), ldo, rows, size, code, _counted(mask, device),
                        _raw_stream(device))
    _wrote(given)
    return out


def dropout_backward(dy, mask, out=None, stream=None):
    """The gradient of ``dropout_forward``: the same map of dy."""
    return dropout_forward(dy, mask, out, stream)


# ---------------------------------------------------------------- layer norm and the residual step
def layer_norm_forward(x, weight=None, bias=None, eps=1e-5, *, out=None, stats=True, stream=None):
    """(y, mean, rstd) of the norm over the last dimension.  mean and rstd are
    what the backward pass takes, and None without ``stats``."""
    args = x, None, weight, bias, eps, None, None, out, stats
    got = _forward(*args) if stream is None else _there(stream, _forward, *args)
    _wrote(out)
    return got[1:]


def residual_norm_forward(x, residual, weight=None, bias=None, eps=1e-5, mask=None, *, out_h=None, out=None,
                          stats=True, stream=None):
    """(h, y, mean, rstd) of h = residual + dropout(x), y = norm(h).  out_h
    may be residual or x (in place)."""
    args = x, residual, weight, bias, eps, mask, out_h, out, stats
    got = _forward(*args) if stream is None else _there(stream, _forward, *args)
    _wrote(out_h, out)
    return got


def _forward(x, residual, weight, bias, eps, mask, h, y, stats):
    device, rows, size, ld, code = _matrix(x, "x")
    wp = bp = None
    wdt = GCLIP_F32
    if bias is not None:
        bp, wdt = _vector(bias, size, x, "bias"), _CODES[bias.dtype]
    if weight is not None:
        wp, wdt = _vector(weight, size, x, "weight"), _CODES[weight.dtype]
        if bias is not None and bias.dtype != weight.dtype:
            raise TypeError("weight and bias must have one dtype")
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        ldy = size
    else:
        ldy = _like(y, x, "out")
    mean = rstd = mp = rp = None
    if stats:
        mean, rstd = torch.empty((2, *x.shape[:-1]), dtype=_F32, device=x.device).unbind(0)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    if residual is None:
        gclip_layernorm_forward(GclipLayerForward(rows, size, code, wdt, eps, x.data_ptr(), ld, None, 0, wp, bp, None,
                                                  0, y.data_ptr(), ldy, mp, rp), _raw_stream(device))
        return None, y, mean, rstd
    ldr = _like(residual, x, "residual")
    if h is None:
        h = torch.empty_like(x, memory_format=torch.contiguous_format)
        ldh = size
    else:
        ldh = _like(h, x, "out_h")
    gclip_residual_forward(GclipLayerForward(rows, size, code, wdt, eps, x.data_ptr(), ld, residual.data_ptr(), ldr,
                                             wp, bp, h.data_ptr(), ldh, y.data_ptr(), ldy, mp, rp),
                           _counted(mask, device) if mask is not None and mask.drops else None, _raw_stream(device))
    return h, y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, dweight=None, dbias=None, accumulate=False,
                        weight_grad=None, bias_grad=None, out=None, stream=None):
    """(dx, dweight, dbias) of the norm of x, from the mean and rstd that its
    forward pass returned.

    dweight, dbias  where the weights' gradients go (binary32 or x's dtype);
                    by default new tensors of weight's dtype
    accumulate      add to them instead (the microbatches' +=)
    weight_grad, bias_grad  whether they are wanted; by default when weight is
                    given, or a buffer for them
    """
    args = dy, None, x, mean, rstd, weight, None, False, dweight, dbias, accumulate, weight_grad, bias_grad, out, None
    dx, _, dw, db = _backward(*args) if stream is None else _there(stream, _backward, *args)
    _wrote(out, dweight, dbias)
    return dx, dw, db


def residual_norm_backward(dy, dh, h, mean, rstd, weight=None, mask=None, *, dweight=None, dbias=None,
                           accumulate=False, weight_grad=None, bias_grad=None, out=None, out_residual=None,
                           stream=None):
    """(dx, dresidual, dweight, dbias) of the residual step, from the h, mean
    and rstd that its forward pass returned and the same mask.  dh is the
    gradient of h from its other uses, or None.  Without dropout dx is
    dresidual, the same tensor.  Otherwise as ``layer_norm_backward``."""
    args = (dy, dh, h, mean, rstd, weight, mask if mask is not None and mask.drops else None, True, dweight, dbias,
            accumulate, weight_grad, bias_grad, out, out_residual)
    got = _backward(*args) if stream is None else _there(stream, _backward, *args)
    _wrote(out, out_residual, dweight, dbias)
    return got


def _backward(dy, dh, x, mean, rstd, weight, mask, residual, dweight, dbias, accumulate, weight_grad, bias_grad, dx,
              dres):
    device, rows, size, ld, code = _matrix(x, "x")
    wp, wdt, gt = None, GCLIP_F32, _F32
    if weight is not None:
        wp, gt = _vector(weight, size, x, "weight"), weight.dtype
        wdt = _CODES[gt]
    want_w = dweight is not None or (weight is not None if weight_grad is None else weight_grad)
    want_b = dbias is not None or (weight is not None if bias_grad is None else bias_grad)
    if accumulate and ((want_w and dweight is None) or (want_b and dbias is None)):
        raise ValueError("accumulate needs the buffers to add to: dweight and dbias")
    mp, rp = _statistic(mean, rows, x, "mean"), _statistic(rstd, rows, x, "rstd")
    lddy, hp, lddh = _like(dy, x, "dy"), None, 0
    if dh is not None:
        hp, lddh = dh.data_ptr(), _like(dh, x, "dh")
    wgp = bgp = None
    nbytes = gclip_layer_workspace(rows, size)
    workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    if want_w or want_b:
        if dweight is not None:
            gt = dweight.dtype
            if dbias is not None and dbias.dtype != gt:
                raise TypeError("dweight and dbias must have one dtype")
        elif dbias is not None:
            gt = dbias.dtype
        if want_w:
            if dweight is None:
                dweight = torch.empty(size, dtype=gt, device=x.device)
            wgp = _vector(dweight, size, x, "dweight")
        if want_b:
            if dbias is None:
                dbias = torch.empty(size, dtype=gt, device=x.device)
            bgp = _vector(dbias, size, x, "dbias")
    second = not residual or mask is not None  # dx apart from dresidual
    if not second:
        if dx is not None and dres is not None and dx is not dres:
            raise ValueError("without dropout dx is dresidual: give one buffer")
        dres = dres if dres is not None else dx
    xp = sp = None
    lddx = ldds = 0
    if second:
        if dx is None:
            dx = torch.empty_like(x, memory_format=torch.contiguous_format)
            lddx = size
        else:
            lddx = _like(dx, x, "out")
        xp = dx.data_ptr()
    if residual:
        if dres is None:
            dres = torch.empty_like(x, memory_format=torch.contiguous_format)
            ldds = size
        else:
            ldds = _like(dres, x, "out_residual")
        sp = dres.data_ptr()
    args = GclipLayerBackward(rows, size, code, wdt, _CODES[gt], 1 if accumulate else 0, dy.data_ptr(), lddy, hp, lddh,
                              x.data_ptr(), ld, mp, rp, wp, sp, ldds, xp, lddx, wgp, bgp, workspace.data_ptr(),
                              nbytes)
    if residual:
        gclip_residual_backward(args, _counted(mask, device) if mask is not None else None, _raw_stream(device))
    else:
        gclip_layernorm_backward(args, _raw_stream(device))
    return dx if second else dres, dres, dweight, dbias


# ---------------------------------------------------------------- under autograd
def _without_tangent(*tensors):
    """Refuse what a forward-mode derivative would be lost of."""
    if _forward_ad._current_level >= 0:
        for t in tensors:
            if t is not None and _forward_ad.unpack_dual(t).tangent is not None:
                raise NotImplementedError("the layers have no forward-mode derivatives")


def _matrix_of(t):
    """A gradient from autograd in a form that the kernels take: an expanded
    or permuted one is copied."""
    _without_tangent(t)
    try:
        _ld(t, "gradient")
        return t
    except ValueError:
        return t.contiguous()


if torch is not None:
    import torch.autograd.forward_ad as _forward_ad
    from torch.autograd.function import once_differentiable

    class _Dropout(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, mask):
            ctx.mask = mask
            return dropout_forward(x, mask)

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            return dropout_backward(_matrix_of(dy), ctx.mask), None

    class _LayerNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, eps):
            y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
            ctx.save_for_backward(x, mean, rstd, weight)
            ctx.bias = (bias.shape, bias.dtype) if bias is not None else None
            return y

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            x, mean, rstd, weight = ctx.saved_tensors
            dw, db = _grad_buffers(ctx, x, weight, 1)
            dx, _, dw, db = _backward(_matrix_of(dy), None, x, mean, rstd, weight, None, False, dw, db, False, False,
                                      False, None, None)
            return dx, dw, db, None

    class _ResidualNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, weight, bias, eps, mask):
            h, y, mean, rstd = residual_norm_forward(x, residual, weight, bias, eps, mask)
            ctx.save_for_backward(h, mean, rstd, weight)
            ctx.bias = (bias.shape, bias.dtype) if bias is not None else None
            ctx.mask = mask
            ctx.set_materialize_grads(False)
            return h, y

        @staticmethod
        @once_differentiable
        def backward(ctx, dh, dy):
            h, mean, rstd, weight = ctx.saved_tensors
            mask = ctx.mask
            dh = _matrix_of(dh) if dh is not None else None
            if not ctx.needs_input_grad[0]:
                mask = None  # dx is not wanted, and dresidual does not depend on it
            if dy is None:  # y is not used: the residual sum alone
                if dh is None:
                    return (None,) * 6
                return dropout_backward(dh, mask) if mask is not None else dh, dh, None, None, None, None
            dw, db = _grad_buffers(ctx, h, weight, 2)
            dx, dres, dw, db = _backward(_matrix_of(dy), dh, h, mean, rstd, weight,
                                         mask if mask is not None and mask.drops else None, True, dw, db, False, False,
                                         False, None, None)
            return dx, dres, dw, db, None, None


def _grad_buffers(ctx, x, weight, at):
    """New buffers for those weights' gradients that are asked for."""
    return (torch.empty(weight.shape, dtype=weight.dtype, device=x.device) if ctx.needs_input_grad[at] else None,
            torch.empty(ctx.bias[0], dtype=ctx.bias[1], device=x.device) if ctx.needs_input_grad[at + 1] else None)


def _tracked(*tensors):
    _without_tangent(*tensors)
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def dropout(x, mask):
    """Dropout of x by the mask (a ``DropoutMask``)."""
    return _Dropout.apply(x, mask) if _tracked(x) else dropout_forward(x, mask)


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """The norm of x over its last dimension."""
    if not _tracked(x, weight, bias):
        return layer_norm_forward(x, weight, bias, eps, stats=False)[0]
    return _LayerNorm.apply(x, weight, bias, eps)


def residual_norm(x, residual, weight=None, bias=None, eps=1e-5, mask=None):
    """(h, y): h = residual + dropout(x), y = the norm of h.  Without a mask
    nothing is dropped (evaluation)."""
    if not _tracked(x, residual, weight, bias):
        return residual_norm_forward(x, residual, weight, bias, eps, mask, stats=False)[:2]
    return _ResidualNorm.apply(x, residual, weight, bias, eps, mask)
