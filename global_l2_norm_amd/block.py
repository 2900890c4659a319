"""The memory-bound operators of a block of the kind that most language models
have now (include/gclip_block.h): RMS norm with the residual's addition, the
(gated) activation, and their 8-bit forms: the norm's output for a product of
8-bit operands, and checkpoints that a backward pass starts from.

As in ``layers`` the functions named like the C ABI take its structures with
raw device addresses, and the others torch tensors:

- ``rms_norm_forward`` / ``_backward``, ``residual_rms_norm_forward`` /
  ``_backward``, ``activation_forward`` / ``_backward``, ``pack8`` and
  ``unpack8`` are the passes themselves, for a program that writes its own
  backward pass.  With ``keep`` a forward pass also leaves what its gradient
  needs in 8 bits (a ``Packed8``), and a backward pass takes that in the place
  of the matrix.
- ``rms_norm``, ``residual_rms_norm`` and ``activation`` are the same under
  autograd, in its backward mode; with ``checkpoint`` they save the 8-bit form
  alone.

Matrices, streams, captures and refusals are those of ``layers``.
"""
import ctypes

try:
    import torch
except ImportError:  # the functions named like the C ABI do without it
    torch = None

from . import _check, _lib
from ._lib import (GCLIP_ACT_GELU, GCLIP_ACT_GELU_TANH, GCLIP_ACT_RELU, GCLIP_ACT_SILU, GCLIP_F32, GCLIP_SCALE_BLOCK,
                   GCLIP_SCALES_BLOCK, GCLIP_SCALES_ROW, GclipPacked8)
from .layers import _counted, _like, _matrix, _there, _vector, _wrote

_byref = ctypes.byref
_pack8, _pack_activate = _lib.PACK_PACKED8.pack, _lib.PACK_ACTIVATE.pack
_pack_forward, _pack_backward = _lib.PACK_RMS_FORWARD.pack, _lib.PACK_RMS_BACKWARD.pack
ACTIVATIONS = {"silu": GCLIP_ACT_SILU, "gelu": GCLIP_ACT_GELU, "gelu_tanh": GCLIP_ACT_GELU_TANH, "relu": GCLIP_ACT_RELU}
_MODES = {"block": GCLIP_SCALES_BLOCK, "row": GCLIP_SCALES_ROW}


# ---------------------------------------------------------------- C ABI names
def _at(args):
    """A structure's address; its bytes are an address to ctypes as they are."""
    return args if type(args) is bytes else _byref(args)


def gclip_rmsnorm_forward(args, stream):
    _check(_lib.lib.gclip_rmsnorm_forward(_at(args), stream), "gclip_rmsnorm_forward")


def gclip_rmsnorm_backward(args, stream):
    _check(_lib.lib.gclip_rmsnorm_backward(_at(args), stream), "gclip_rmsnorm_backward")


def gclip_residual_rms_forward(args, drop, stream):
    _check(_lib.lib.gclip_residual_rms_forward(_at(args), _byref(drop) if drop is not None else None, stream),
           "gclip_residual_rms_forward")


def gclip_residual_rms_backward(args, drop, stream):
    _check(_lib.lib.gclip_residual_rms_backward(_at(args), _byref(drop) if drop is not None else None, stream),
           "gclip_residual_rms_backward")


def gclip_rms_workspace(rows, size):
    return _lib.lib.gclip_rms_workspace(rows, size)


def gclip_activation_forward(args, stream):
    _check(_lib.lib.gclip_activation_forward(_at(args), stream), "gclip_activation_forward")


def gclip_activation_backward(args, stream):
    _check(_lib.lib.gclip_activation_backward(_at(args), stream), "gclip_activation_backward")


def gclip_pack(x, ldx, out, rows, size, dtype, stream):
    _check(_lib.lib.gclip_pack(x, ldx, _at(out), rows, size, dtype, stream), "gclip_pack")


def gclip_unpack(x, out, ldout, rows, size, dtype, stream):
    _check(_lib.lib.gclip_unpack(_at(x), out, ldout, rows, size, dtype, stream), "gclip_unpack")


# ---------------------------------------------------------------- matrices in 8 bits
if torch is not None:
    from .layers import _CODES, _F32, _raw_stream
    _E4M3 = torch.float8_e4m3fn
    # a size in a tuple costs 0.7 us more than one in arguments
    _empty, _empty_like, _contiguous = torch.empty, torch.empty_like, torch.contiguous_format
_NONE8 = (0, 0, 0, 0, 0)


class Packed8:
    """A matrix in 8 bits: it stands for ``values * scales``, a scale for each
    128 columns of a row ("block") or for the row.

    values   torch.float8_e4m3fn, the matrix's shape; its rows begin at
             multiples of 8 bytes, and the bytes from a row's end to the next
             multiple belong to it (``values`` is a view without them)
    scales   torch.float32, contiguous, [..., scales of a row]

    ``pack8``, and the forward passes' ``keep`` and ``packed``, make them.
    """

    __slots__ = ("held", "size", "scales", "fields")

    def __init__(self, values, scales):
        if values.dtype != _E4M3 or scales.dtype != _F32:
            raise TypeError(f"values must be float8_e4m3fn and scales float32, not {values.dtype} and {scales.dtype}")
        shape = values.shape
        if not shape or scales.shape[:-1] != shape[:-1] or not scales.shape or not scales.is_contiguous():
            raise ValueError("scales must be contiguous, [..., scales of a row] of values [..., columns]")
        size, count = shape[-1], scales.shape[-1]
        if count == -(-size // GCLIP_SCALE_BLOCK):
            mode = GCLIP_SCALES_BLOCK
        elif count == 1:
            mode = GCLIP_SCALES_ROW
        else:
            raise ValueError(f"{count} scales a row for {size} columns: one, or one for each {GCLIP_SCALE_BLOCK}")
        if scales.get_device() != values.get_device():
            raise ValueError("values and scales must be on one device")
        self.held, self.size, self.scales = values, size, scales
        self.fields = values.data_ptr(), _row_bytes(values), scales.data_ptr(), mode, 0

    @classmethod
    def _new(cls, x, size, mode):
        """Memory for x in 8 bits; the device's allocator aligns it."""
        self = cls.__new__(cls)
        lead = x.shape[:-1]
        ld = (size + 7) // 8 * 8
        if ld == size:
            held = _empty_like(x, dtype=_E4M3, memory_format=_contiguous)
        else:
            held = _empty(*lead, ld, dtype=_E4M3, device=x.device)
        scales = _empty(*lead, 1 if mode else (size + 127) // GCLIP_SCALE_BLOCK, dtype=_F32, device=x.device)
        self.held, self.size, self.scales = held, size, scales
        # a row of one block has one scale either way, which is a block's to a reader
        self.fields = held.data_ptr(), ld, scales.data_ptr(), mode if size > GCLIP_SCALE_BLOCK else GCLIP_SCALES_BLOCK, 0
        return self

    @property
    def values(self):
        held, size = self.held, self.size
        return held if held.shape[-1] == size else held[..., :size]

    def __reduce__(self):
        return Packed8, (self.values, self.scales)

    @property
    def args(self):
        """The C ABI's structure."""
        return GclipPacked8(*self.fields)

    @property
    def shape(self):
        shape = self.held.shape
        return shape if shape[-1] == self.size else torch.Size((*shape[:-1], self.size))

    @property
    def device(self):
        return self.held.device

    def record_stream(self, stream):
        self.held.record_stream(stream)
        self.scales.record_stream(stream)

    def dequantize(self):
        """The values that it stands for, in binary32."""
        return unpack8(self, _F32)


def _row_bytes(values):
    """Distance of the rows of a Packed8's values; what lies behind each row's
    end up to a multiple of eight has to be the storage's."""
    shape, stride = values.shape, values.stride()
    size = shape[-1]
    rows = values.numel() // size if size else 0
    if size > 1 and stride[-1] != 1:
        raise ValueError("values: the last dimension must be adjacent in memory")
    lead = [(n, s) for n, s in zip(shape[:-1], stride[:-1]) if n != 1]
    if any(a[1] != b[0] * b[1] for a, b in zip(lead, lead[1:])):
        raise ValueError("values: the rows must lie at one distance")
    whole = (size + 7) // 8 * 8
    ld = lead[-1][1] if lead else whole
    if rows == 0:
        return whole
    if values.data_ptr() % 8 or ld % 8 or ld < 0:
        raise ValueError("values: rows must begin at multiples of 8 bytes")
    last = values.storage_offset() + (rows - 1) * ld + whole
    if last > values.untyped_storage().nbytes():
        raise ValueError("values: the last row needs its bytes up to a multiple of 8")
    return ld


def _packed(p, x, name):
    """A Packed8 of x's shape and device."""
    if not isinstance(p, Packed8):
        raise TypeError(f"{name} must be a Packed8 or a tensor, not {type(p).__name__}")
    if p.shape != x.shape or p.held.get_device() != x.get_device():
        raise ValueError(f"{name} must have shape {tuple(x.shape)} on {x.device}")
    fields = p.fields
    if p.held.data_ptr() != fields[0] or p.scales.data_ptr() != fields[2]:
        raise ValueError(f"{name} has another storage than when it was made")
    return fields


def _blocks(p, x, name):
    """The same with a scale for each block, as the activation's gradient takes
    them."""
    fields = _packed(p, x, name)
    if fields[3] != GCLIP_SCALES_BLOCK:
        raise ValueError(f"{name} must have a scale for each {GCLIP_SCALE_BLOCK} columns (\"block\"), not one a row")
    return fields


def _mode(name):
    try:
        return _MODES[name]
    except KeyError:
        raise ValueError(f'scales must be "block" or "row", not {name!r}') from None


def _there8(stream, f, *args):
    for t in args:
        if isinstance(t, Packed8):
            t.record_stream(stream)
    return _there(stream, f, *args)


def pack8(x, scales="block", *, stream=None):
    """x in 8 bits (a ``Packed8``), with a scale for each 128 columns of a row
    ("block") or for each row ("row")."""
    if stream is not None:
        return _there8(stream, pack8, x, scales)
    mode = _mode(scales)
    device, rows, size, ld, code = _matrix(x, "x")
    if size == 0:
        raise ValueError("x must have at least one column")
    out = Packed8._new(x, size, mode)
    gclip_pack(x.data_ptr(), ld, _pack8(*out.fields), rows, size, code, _raw_stream(device))
    return out


def unpack8(packed, dtype=None, *, out=None, stream=None):
    """The matrix that a ``Packed8`` stands for, in ``dtype`` (by default
    out's, or bfloat16)."""
    if stream is not None:
        return _there8(stream, _unpack8, packed, dtype, out)
    return _unpack8(packed, dtype, out)


def _unpack8(packed, dtype, out):
    if not isinstance(packed, Packed8):
        raise TypeError(f"packed must be a Packed8, not {type(packed).__name__}")
    if out is None:
        new = _empty(*packed.shape, dtype=dtype or torch.bfloat16, device=packed.device)
    elif dtype is not None and out.dtype != dtype:
        raise TypeError(f"out must have dtype {dtype}, not {out.dtype}")
    else:
        new = out
    device, rows, size, ld, code = _matrix(new, "out")
    gclip_unpack(_pack8(*_packed(packed, new, "packed")), new.data_ptr(), ld, rows, size, code, _raw_stream(device))
    _wrote(out)
    return new


# ---------------------------------------------------------------- RMS norm and its residual step
def rms_norm_forward(x, weight=None, eps=1e-6, *, out=None, packed=None, keep=False, stats=True, stream=None):
    """(y, rstd, kept) of the norm over the last dimension.

    packed  "row" or "block": y in 8 bits (a ``Packed8``) with such scales, for
            a product of 8-bit operands
    keep    also x in 8 bits (``kept``, else None), which ``rms_norm_backward``
            takes in the place of x
    stats   rstd is what the backward pass takes, and None without
    """
    args = x, None, weight, eps, None, None, out, packed, keep, stats
    got = _forward(*args) if stream is None else _there(stream, _forward, *args)
    _wrote(out)
    return got[1:]


def residual_rms_norm_forward(x, residual, weight=None, eps=1e-6, mask=None, *, out_h=None, out=None, packed=None,
                              keep=False, stats=True, stream=None):
    """(h, y, rstd, kept) of h = residual + dropout(x), y = norm(h); kept is of
    h.  out_h may be residual or x (in place).  Otherwise as
    ``rms_norm_forward``."""
    args = x, residual, weight, eps, mask, out_h, out, packed, keep, stats
    got = _forward(*args) if stream is None else _there(stream, _forward, *args)
    _wrote(out_h, out)
    return got


def _forward(x, residual, weight, eps, mask, h, y, packed, keep, stats):
    device, rows, size, ld, code = _matrix(x, "x")
    wp, wdt = 0, GCLIP_F32
    if weight is not None:
        wp, wdt = _vector(weight, size, x, "weight"), _CODES[weight.dtype]
    yp, ldy, y8 = 0, 0, _NONE8
    if packed is not None:
        if y is not None:
            raise ValueError("out is for a y that is not packed")
        mode = _mode(packed)
        y = Packed8._new(x, size, mode)
        # the scale of a row comes with its sum, and rounds otherwise than a block's
        y8 = y.fields if size > GCLIP_SCALE_BLOCK else (*y.fields[:3], mode, 0)
    elif y is None:
        y = _empty_like(x, memory_format=_contiguous)
        yp, ldy = y.data_ptr(), size
    else:
        ldy = _like(y, x, "out")
        yp = y.data_ptr()
    kept, k8 = None, _NONE8
    if keep:
        kept = Packed8._new(x, size, GCLIP_SCALES_BLOCK)
        k8 = kept.fields
    rstd, rp = None, 0
    if stats:
        lead = x.shape[:-1]
        rstd = _empty(*lead, dtype=_F32, device=x.device) if lead else _empty((), dtype=_F32, device=x.device)
        rp = rstd.data_ptr()
    if residual is None:
        gclip_rmsnorm_forward(_pack_forward(rows, size, code, wdt, float(eps), x.data_ptr(), ld, 0, 0, wp, 0, 0, yp, ldy,
                                            *y8, *k8, rp), _raw_stream(device))
        return None, y, rstd, kept
    ldr = _like(residual, x, "residual")
    if h is None:
        h = _empty_like(x, memory_format=_contiguous)
        ldh = size
    else:
        ldh = _like(h, x, "out_h")
    gclip_residual_rms_forward(_pack_forward(rows, size, code, wdt, float(eps), x.data_ptr(), ld, residual.data_ptr(), ldr,
                                             wp, h.data_ptr(), ldh, yp, ldy, *y8, *k8, rp),
                               _counted(mask, device) if mask is not None and mask.drops else None,
                               _raw_stream(device))
    return h, y, rstd, kept


def rms_norm_backward(dy, x, rstd, weight=None, *, dweight=None, accumulate=False, weight_grad=None, out=None,
                      stream=None):
    """(dx, dweight) of the norm of x, from the rstd that its forward pass
    returned.  x may be what that pass kept in 8 bits.

    dweight      where the weight's gradient goes (binary32 or dy's dtype); by
                 default a new tensor of weight's dtype
    accumulate   add to it instead (the microbatches' +=)
    weight_grad  whether it is wanted; by default when weight is given, or a
                 buffer for it
    """
    args = dy, None, x, rstd, weight, None, False, dweight, accumulate, weight_grad, out, None
    dx, _, dw = _backward(*args) if stream is None else _there8(stream, _backward, *args)
    _wrote(out, dweight)
    return dx, dw


def residual_rms_norm_backward(dy, dh, h, rstd, weight=None, mask=None, *, dweight=None, accumulate=False,
                               weight_grad=None, out=None, out_residual=None, stream=None):
    """(dx, dresidual, dweight) of the residual step, from the h (or its 8-bit
    form) and rstd that its forward pass returned and the same mask.  dh is the
    gradient of h from its other uses, or None.  Without dropout dx is
    dresidual, the same tensor.  Otherwise as ``rms_norm_backward``."""
    args = (dy, dh, h, rstd, weight, mask if mask is not None and mask.drops else None, True, dweight, accumulate,
            weight_grad, out, out_residual)
    got = _backward(*args) if stream is None else _there8(stream, _backward, *args)
    _wrote(out, out_residual, dweight)
    return got


def _backward(dy, dh, x, rstd, weight, mask, residual, dweight, accumulate, weight_grad, dx, dres):
    device, rows, size, lddy, code = _matrix(dy, "dy")
    wp, wdt, gt = 0, GCLIP_F32, _F32
    if weight is not None:
        wp, gt = _vector(weight, size, dy, "weight"), weight.dtype
        wdt = _CODES[gt]
    want = dweight is not None or (weight is not None if weight_grad is None else weight_grad)
    if accumulate and want and dweight is None:
        raise ValueError("accumulate needs the buffer to add to: dweight")
    if rstd.dtype != _F32:
        raise TypeError(f"rstd must be float32, not {rstd.dtype}")
    rp = _vector(rstd, rows, dy, "rstd")
    xp, ldx, x8 = 0, 0, _NONE8
    if isinstance(x, Packed8):
        x8 = _packed(x, dy, "x")
    else:
        ldx = _like(x, dy, "x")
        xp = x.data_ptr()
    hp, lddh = 0, 0
    if dh is not None:
        hp, lddh = dh.data_ptr(), _like(dh, dy, "dh")
    nbytes = gclip_rms_workspace(rows, size)
    workspace = _empty(nbytes, dtype=torch.uint8, device=dy.device) if nbytes else None
    wgp = 0
    if want:
        if dweight is None:
            dweight = _empty(size, dtype=gt, device=dy.device)
        gt = dweight.dtype
        wgp = _vector(dweight, size, dy, "dweight")
    second = not residual or mask is not None  # dx apart from dresidual
    if not second:
        if dx is not None and dres is not None and dx is not dres:
            raise ValueError("without dropout dx is dresidual: give one buffer")
        dres = dres if dres is not None else dx
    dxp = sp = lddx = ldds = 0
    if second:
        if dx is None:
            dx = _empty_like(dy, memory_format=_contiguous)
            lddx = size
        else:
            lddx = _like(dx, dy, "out")
        dxp = dx.data_ptr()
    if residual:
        if dres is None:
            dres = _empty_like(dy, memory_format=_contiguous)
            ldds = size
        else:
            ldds = _like(dres, dy, "out_residual")
        sp = dres.data_ptr()
    args = _pack_backward(rows, size, code, wdt, _CODES[gt], 1 if accumulate else 0, dy.data_ptr(), lddy, hp, lddh, xp,
                          ldx, *x8, rp, wp, sp, ldds, dxp, lddx, wgp, workspace.data_ptr() if nbytes else 0, nbytes)
    if residual:
        gclip_residual_rms_backward(args, _counted(mask, device) if mask is not None else None, _raw_stream(device))
    else:
        gclip_rmsnorm_backward(args, _raw_stream(device))
    return dx if second else dres, dres, dweight


# ---------------------------------------------------------------- the activation
def activation_forward(gate, up=None, kind="silu", *, keep=False, out=None, stream=None):
    """(y, gate8, up8): y = act(gate) * up, or act(gate) without up.  kind is
    "silu", "gelu", "gelu_tanh" or "relu".  With ``keep`` gate8 and up8 are
    both in 8 bits, which ``activation_backward`` takes in their place; else
    None."""
    args = gate, up, kind, keep, out
    got = _activation_forward(*args) if stream is None else _there(stream, _activation_forward, *args)
    _wrote(out)
    return got


def _kind(name):
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"kind must be one of {', '.join(ACTIVATIONS)}, not {name!r}") from None


def _activation_forward(gate, up, kind, keep, y):
    kind = _kind(kind)
    device, rows, size, ld, code = _matrix(gate, "gate")
    up_at, ldu = (up.data_ptr(), _like(up, gate, "up")) if up is not None else (0, 0)
    if y is None:
        y = _empty_like(gate, memory_format=_contiguous)
        ldy = size
    else:
        ldy = _like(y, gate, "out")
    gate8 = up8 = None
    if keep:
        gate8 = Packed8._new(gate, size, GCLIP_SCALES_BLOCK)
        if up is not None:
            up8 = Packed8._new(gate, size, GCLIP_SCALES_BLOCK)
    if rows == 0 or size == 0:
        return y, gate8, up8
    gclip_activation_forward(_pack_activate(rows, size, code, kind, gate.data_ptr(), ld, up_at, ldu,
                                            *(gate8.fields if keep else _NONE8),
                                            *(up8.fields if up8 is not None else _NONE8), y.data_ptr(), ldy, 0, 0, 0, 0,
                                            0, 0), _raw_stream(device))
    return y, gate8, up8


def activation_backward(dy, gate, up=None, kind="silu", *, recompute=False, out=None, out_gate=None, out_up=None,
                        stream=None):
    """(dgate, dup, y) of ``activation_forward``, from gate and up or from what
    it kept of both in 8 bits.  dup is None without up.  y is computed again
    with ``recompute`` (for the weight's gradient of the product behind it),
    else None."""
    args = dy, gate, up, kind, recompute, out, out_gate, out_up
    got = _activation_backward(*args) if stream is None else _there8(stream, _activation_backward, *args)
    _wrote(out, out_gate, out_up)
    return got


def _activation_backward(dy, gate, up, kind, recompute, y, dgate, dup):
    kind = _kind(kind)
    device, rows, size, lddy, code = _matrix(dy, "dy")
    eight = isinstance(gate, Packed8)
    if up is not None and isinstance(up, Packed8) != eight:
        raise TypeError("gate and up must both be tensors, or both in 8 bits")
    gp = up_at = ldg = ldu = 0
    g8 = u8 = _NONE8
    if eight:
        g8 = _blocks(gate, dy, "gate")
        if up is not None:
            u8 = _blocks(up, dy, "up")
    else:
        ldg = _like(gate, dy, "gate")
        gp = gate.data_ptr()
        if up is not None:
            ldu = _like(up, dy, "up")
            up_at = up.data_ptr()
    if dgate is None:
        dgate = _empty_like(dy, memory_format=_contiguous)
        lddg = size
    else:
        lddg = _like(dgate, dy, "out_gate")
    dup_at = lddu = 0
    if up is not None:
        if dup is None:
            dup = _empty_like(dy, memory_format=_contiguous)
            lddu = size
        else:
            lddu = _like(dup, dy, "out_up")
        dup_at = dup.data_ptr()
    elif dup is not None:
        raise ValueError("out_up is for a gated activation")
    yp = ldy = 0
    if y is not None and not recompute:
        raise ValueError("out is for recompute")
    if recompute:
        if y is None:
            y = _empty_like(dy, memory_format=_contiguous)
            ldy = size
        else:
            ldy = _like(y, dy, "out")
        yp = y.data_ptr()
    if rows and size:
        gclip_activation_backward(_pack_activate(rows, size, code, kind, gp, ldg, up_at, ldu, *g8, *u8, yp, ldy,
                                                 dy.data_ptr(), lddy, dgate.data_ptr(), lddg, dup_at, lddu),
                                  _raw_stream(device))
    return dgate, dup, y


# ---------------------------------------------------------------- under autograd
if torch is not None:
    from torch.autograd.function import once_differentiable

    from .layers import _matrix_of, _tracked, dropout_backward

    def _of_held(held, scales, size):
        """A Packed8 from the memory that holds its rows whole, which is what
        autograd saves: a hook that moves a saved tensor keeps its values and
        not its layout."""
        return Packed8(held if held.shape[-1] == size else held[..., :size], scales)

    def _save(ctx, kept, x, *more):
        """x or its 8-bit form, for the backward pass."""
        ctx.packed = kept is not None
        ctx.size = x.shape[-1]
        ctx.save_for_backward(*((kept.held, kept.scales) if kept is not None else (x, None)), *more)

    def _saved(ctx):
        a, b, *more = ctx.saved_tensors
        return _of_held(a, b, ctx.size) if ctx.packed else a, *more

    class _RmsNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, eps, checkpoint):
            y, rstd, kept = rms_norm_forward(x, weight, eps, keep=checkpoint)
            _save(ctx, kept, x, rstd, weight)
            return y

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            x, rstd, weight = _saved(ctx)
            dw = _grad_buffer(ctx, weight, 1)
            dx, _, dw = _backward(_matrix_of(dy), None, x, rstd, weight, None, False, dw, False, False, None, None)
            return dx, dw, None, None

    class _ResidualRmsNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, weight, eps, mask, checkpoint):
            h, y, rstd, kept = residual_rms_norm_forward(x, residual, weight, eps, mask, keep=checkpoint)
            _save(ctx, kept, h, rstd, weight)
            ctx.mask = mask
            ctx.set_materialize_grads(False)
            return h, y

        @staticmethod
        @once_differentiable
        def backward(ctx, dh, dy):
            h, rstd, weight = _saved(ctx)
            mask = ctx.mask
            dh = _matrix_of(dh) if dh is not None else None
            if not ctx.needs_input_grad[0]:
                mask = None  # dx is not wanted, and dresidual does not depend on it
            if dy is None:  # y is not used: the residual sum alone
                if dh is None:
                    return (None,) * 6
                return dropout_backward(dh, mask) if mask is not None else dh, dh, None, None, None, None
            dw = _grad_buffer(ctx, weight, 2)
            dx, dres, dw = _backward(_matrix_of(dy), dh, h, rstd, weight,
                                     mask if mask is not None and mask.drops else None, True, dw, False, False, None,
                                     None)
            return dx, dres, dw, None, None, None

    class _Activation(torch.autograd.Function):
        @staticmethod
        def forward(ctx, gate, up, kind, checkpoint):
            y, gate8, up8 = activation_forward(gate, up, kind, keep=checkpoint)
            ctx.kind, ctx.packed, ctx.gated, ctx.size = kind, checkpoint, up is not None, gate.shape[-1]
            if checkpoint:
                ctx.save_for_backward(gate8.held, gate8.scales, *((up8.held, up8.scales) if up is not None else ()))
            else:
                ctx.save_for_backward(gate, *((up,) if up is not None else ()))
            return y

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            saved = ctx.saved_tensors
            if ctx.packed:
                saved = [_of_held(*saved[i:i + 2], ctx.size) for i in range(0, len(saved), 2)]
            dgate, dup, _ = activation_backward(_matrix_of(dy), saved[0], saved[1] if ctx.gated else None, ctx.kind)
            return dgate, dup, None, None


def _grad_buffer(ctx, weight, at):
    """A new buffer for the weight's gradient, if it is asked for."""
    return torch.empty(weight.shape, dtype=weight.dtype, device=weight.device) if ctx.needs_input_grad[at] else None


def rms_norm(x, weight=None, eps=1e-6, *, checkpoint=False):
    """The RMS norm of x over its last dimension.  With ``checkpoint`` the
    backward pass keeps x in 8 bits alone, and starts from that."""
    if not _tracked(x, weight):
        return rms_norm_forward(x, weight, eps, stats=False)[0]
    return _RmsNorm.apply(x, weight, eps, checkpoint)


def residual_rms_norm(x, residual, weight=None, eps=1e-6, mask=None, *, checkpoint=False):
    """(h, y): h = residual + dropout(x), y = the RMS norm of h.  Without a
    mask nothing is dropped (evaluation).  checkpoint: as in ``rms_norm``, of
    h."""
    if not _tracked(x, residual, weight):
        return residual_rms_norm_forward(x, residual, weight, eps, mask, stats=False)[:2]
    return _ResidualRmsNorm.apply(x, residual, weight, eps, mask, checkpoint)


def activation(gate, up=None, kind="silu", *, checkpoint=False):
    """act(gate) * up, or act(gate) without up.  With ``checkpoint`` the
    backward pass keeps gate and up in 8 bits alone, and starts from that.

    The gradients of gate and up are two tensors.  Where both are halves of one
    product's output, torch then puts them together, which takes longer than
    the kernels; a backward pass of one's own writes both halves at once
    (``activation_backward``'s out_gate and out_up)."""
    if not _tracked(gate, up):
        return activation_forward(gate, up, kind)[0]
    return _Activation.apply(gate, up, kind, checkpoint)
