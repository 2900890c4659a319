"""Log probabilities of given tokens, with the entropy and the likeliest
alternatives, and their gradient (include/gclip_logprob.h): the loss that the
backward pass starts from, and what a server answers with.

``token_log_probs_forward`` / ``_backward`` are the passes themselves,
``token_log_probs`` is the same under autograd, in its backward mode.
Matrices, streams, captures and refusals are those of ``layers``.
"""
from operator import index
from typing import NamedTuple

try:
    import torch
except ImportError:  # the functions named like the C ABI do without it
    torch = None

from . import _check, _lib
from ._lib import GCLIP_LOGPROB_MAX_TOP
from .block import _at
from .layers import _like, _matrix, _there, _vector, _wrote

_pack = _lib.PACK_LOGPROBS.pack


# ---------------------------------------------------------------- C ABI names
def gclip_logprob_forward(args, stream):
    _check(_lib.lib.gclip_logprob_forward(_at(args), stream), "gclip_logprob_forward")


def gclip_logprob_backward(args, stream):
    _check(_lib.lib.gclip_logprob_backward(_at(args), stream), "gclip_logprob_backward")


def gclip_logprob_workspace(rows, size, top):
    return _lib.lib.gclip_logprob_workspace(rows, size, top)


# ---------------------------------------------------------------- the passes
if torch is not None:
    from .layers import _F32, _raw_stream
    _I64 = torch.int64
    _empty = torch.empty


class TokenLogProbs(NamedTuple):
    """What ``token_log_probs_forward`` returns; what was not asked for is
    None.  logp and entropy have the shape of the logits without their last
    dimension, the others one more: of 2 (the largest logit m, and the
    logarithm of the sum of e^(x - m)), and of the alternatives."""

    logp: object
    entropy: object
    stats: object
    top_logp: object
    top_ids: object


def _targets(t, rows, x):
    if t.dtype != _I64:
        raise TypeError(f"targets must be int64, not {t.dtype}")
    if t.numel() != rows or not t.is_contiguous() or t.get_device() != x.get_device():
        raise ValueError(f"targets must hold {rows} contiguous elements on {x.device}")
    return t.data_ptr()


def _ignored(i):
    i = index(i)
    if not -1 << 63 <= i < 1 << 63:
        raise ValueError(f"ignore_index must be an int64, not {i}")
    return i


def _numbers(t, rows, x, name):
    if t.dtype != _F32:
        raise TypeError(f"{name} must be float32, not {t.dtype}")
    return _vector(t, rows, x, name)


def token_log_probs_forward(logits, targets=None, *, entropy=False, top=0, ignore_index=-100, stats=True, stream=None):
    """A ``TokenLogProbs`` of logits [..., tokens].

    targets       int64, one token of each row; None: no logp
    entropy       whether the entropy of each row is wanted
    top           how many alternatives (up to 32): their log probabilities,
                  largest first, and tokens, of equal ones the lowest first
    ignore_index  the target of rows that count for nothing: zeros, and
                  alternatives -1 with log probabilities of -infinity
    stats         they are what the backward pass takes, and None without
    """
    args = logits, targets, entropy, top, ignore_index, stats
    return _forward(*args) if stream is None else _there(stream, _forward, *args)


def _forward(logits, targets, entropy, top, ignore, stats):
    device, rows, size, ld, code = _matrix(logits, "logits")
    if not 0 <= top <= min(GCLIP_LOGPROB_MAX_TOP, size):
        raise ValueError(f"top must be at most {GCLIP_LOGPROB_MAX_TOP} and the {size} tokens, not {top}")
    lead = logits.shape[:-1]
    tp = _targets(targets, rows, logits) if targets is not None else 0
    on = logits.device
    row = lead or ((),)  # a size in a tuple costs 0.7 us more than one in arguments
    logp = _empty(*row, dtype=_F32, device=on) if targets is not None else None
    stats = _empty(*lead, 2, dtype=_F32, device=on) if stats else None
    h = _empty(*row, dtype=_F32, device=on) if entropy else None
    top_logp = top_ids = None
    if top:
        top_logp, top_ids = _empty(*lead, top, dtype=_F32, device=on), _empty(*lead, top, dtype=_I64, device=on)
    nbytes = gclip_logprob_workspace(rows, size, top)
    workspace = _empty(nbytes, dtype=torch.uint8, device=on) if nbytes else None
    at = lambda t: t.data_ptr() if t is not None else 0  # noqa: E731
    gclip_logprob_forward(_pack(rows, size, code, top, logits.data_ptr(), ld, tp, _ignored(ignore), at(stats), at(logp),
                                at(h), at(top_logp), at(top_ids), 0, 0, 0, 0, at(workspace), nbytes), _raw_stream(device))
    return TokenLogProbs(logp, h, stats, top_logp, top_ids)


def token_log_probs_backward(dlogp, dentropy, logits, targets, stats, entropy=None, *, ignore_index=-100, out=None,
                             stream=None):
    """The gradient of the logits from those of logp and of the entropy (None:
    not used), and the stats and entropy that the forward pass returned.  out may
    be logits."""
    args = dlogp, dentropy, logits, targets, stats, entropy, ignore_index, out
    got = _backward(*args) if stream is None else _there(stream, _backward, *args)
    _wrote(out)
    return got


def _backward(dlogp, dentropy, logits, targets, stats, entropy, ignore, out):
    device, rows, size, ld, code = _matrix(logits, "logits")
    tp, sp = _targets(targets, rows, logits), _numbers(stats, 2 * rows, logits, "stats")
    dp = _numbers(dlogp, rows, logits, "dlogp")
    ep = hp = 0
    if dentropy is not None:
        if entropy is None:
            raise ValueError("dentropy needs the entropy of the forward pass")
        ep, hp = _numbers(dentropy, rows, logits, "dentropy"), _numbers(entropy, rows, logits, "entropy")
    if out is None:
        out = torch.empty_like(logits, memory_format=torch.contiguous_format)
        ldo = size
    else:
        ldo = _like(out, logits, "out")
    gclip_logprob_backward(_pack(rows, size, code, 0, logits.data_ptr(), ld, tp, _ignored(ignore), sp, 0, hp, 0, 0, dp,
                                 ep, out.data_ptr(), ldo, 0, 0), _raw_stream(device))
    return out


# ---------------------------------------------------------------- under autograd
if torch is not None:
    from torch.autograd.function import once_differentiable

    from .layers import _tracked, _without_tangent

    class _TokenLogProbs(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, targets, entropy, top, ignore):
            r = token_log_probs_forward(logits, targets, entropy=entropy, top=top, ignore_index=ignore)
            ctx.save_for_backward(logits, targets, r.stats, r.entropy)
            ctx.ignore = ignore
            ctx.set_materialize_grads(False)
            ctx.mark_non_differentiable(*(t for t in (r.stats, r.top_logp, r.top_ids) if t is not None))
            return tuple(r)

        @staticmethod
        @once_differentiable
        def backward(ctx, dlogp, dentropy, *_):
            if dlogp is None and dentropy is None:
                return (None,) * 5
            _without_tangent(dlogp, dentropy)
            logits, targets, stats, entropy = ctx.saved_tensors
            dlogp = torch.zeros_like(stats[..., 0]) if dlogp is None else dlogp.contiguous()
            dentropy = dentropy.contiguous() if dentropy is not None else None
            return _backward(dlogp, dentropy, logits, targets, stats, entropy, ctx.ignore, None), None, None, None, None


def token_log_probs(logits, targets, *, entropy=False, top=0, ignore_index=-100):
    """A ``TokenLogProbs`` whose logp and entropy have gradients; the others
    have none.  Without targets there are none: ``token_log_probs_forward``."""
    if targets is None:
        raise TypeError("token_log_probs needs targets; token_log_probs_forward does without")
    targets = targets.contiguous()
    if not _tracked(logits):
        return token_log_probs_forward(logits, targets, entropy=entropy, top=top, ignore_index=ignore_index)
    return TokenLogProbs(*_TokenLogProbs.apply(logits, targets, entropy, top, ignore_index))
