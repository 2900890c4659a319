"""The layer calls of the C ABI on the CPU: argument errors come back before
any GPU work.  No call here has valid arguments and rows at once, but for the
ones of the overlap test, which runs only where there is no GPU to reach."""
import ctypes

import pytest

from global_l2_norm_amd import _lib

L = _lib.lib
OK, EINVAL, EDTYPE = _lib.GCLIP_OK, _lib.GCLIP_EINVAL, _lib.GCLIP_EDTYPE
F32, F16, BF16 = _lib.GCLIP_F32, _lib.GCLIP_F16, _lib.GCLIP_BF16
MOST = 0x7ffffff0


def fwd(**over):
    a = dict(rows=4, size=16, dtype=F32, weight_dtype=F32, eps=1e-5, x=0x10000, ldx=16, residual=None, ldresidual=0,
             weight=0x1000, bias=0x2000, h=None, ldh=0, y=0x20000, ldy=16, mean=0x3000, rstd=0x4000)
    a.update(over)
    return _lib.GclipLayerForward(**a)


def bwd(**over):
    a = dict(rows=4, size=16, dtype=F32, weight_dtype=F32, grad_dtype=F32, accumulate=0, dy=0x10000, lddy=16, dh=None,
             lddh=0, x=0x20000, ldx=16, mean=0x3000, rstd=0x4000, weight=0x1000, dresidual=None, lddresidual=0,
             dx=0x30000, lddx=16, dweight=0x5000, dbias=0x6000, workspace=0x100000, workspace_bytes=1 << 20)
    a.update(over)
    return _lib.GclipLayerBackward(**a)


RES_F = dict(residual=0x30000, ldresidual=16, h=0x40000, ldh=16)
RES_B = dict(dh=0x40000, lddh=16, dresidual=0x50000, lddresidual=16)


def drop(p=0.5, **over):
    a = dict(p=p, seed=1, step=0, site=0, d_step=None)
    a.update(over)
    return _lib.GclipDropout(**a)


BAD_BOTH = [
    (dict(rows=-1), EINVAL), (dict(rows=MOST + 1), EINVAL), (dict(size=0), EINVAL), (dict(size=-3), EINVAL),
    (dict(size=MOST + 1), EINVAL), (dict(dtype=3), EDTYPE), (dict(dtype=-1), EDTYPE), (dict(weight_dtype=F16), EDTYPE),
    (dict(dtype=BF16, weight_dtype=F16), EDTYPE), (dict(x=None), EINVAL), (dict(x=0x10002), EINVAL),
    (dict(ldx=-16), EINVAL), (dict(ldx=1 << 60), EINVAL), (dict(mean=0x3002), EINVAL), (dict(weight=0x1001), EINVAL),
]


@pytest.mark.parametrize("over,code", BAD_BOTH + [
    (dict(eps=0.0), EINVAL), (dict(eps=-1e-5), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(eps=float("inf")), EINVAL), (dict(eps=1e39), EINVAL), (dict(eps=1e-39), EINVAL),
    (dict(y=None), EINVAL), (dict(y=0x20001), EINVAL), (dict(ldy=15), EINVAL), (dict(ldy=0), EINVAL),
    (dict(bias=0x2002), EINVAL), (dict(mean=None), EINVAL), (dict(rstd=None), EINVAL),
    (dict(residual=0x30000), EINVAL), (dict(h=0x40000), EINVAL),
    (dict(y=0x10040), EINVAL),                    # y a row behind x
    (dict(y=0x10000, ldy=32), EINVAL),            # in place, other ld
    (dict(ldx=0, y=0x10000), EINVAL),             # over a broadcast row
    (dict(mean=0x20010), EINVAL),                 # mean inside y
    (dict(rstd=0x3004), EINVAL),                  # rstd over mean
    (dict(y=0x1000 - 64 * 3), EINVAL),            # y's last row over weight
])
def test_norm_forward_refuses(over, code):
    assert L.gclip_layernorm_forward(fwd(**over), None) == code


@pytest.mark.parametrize("over,code", [
    (dict(residual=None), EINVAL), (dict(h=None), EINVAL), (dict(ldh=8), EINVAL), (dict(ldresidual=-1), EINVAL),
    (dict(h=0x20000), EINVAL),                    # h and y in one place
    (dict(h=0x30010), EINVAL),                    # h a few columns off residual
])
def test_residual_forward_refuses(over, code):
    assert L.gclip_residual_forward(fwd(**{**RES_F, **over}), None, None) == code


@pytest.mark.parametrize("over,code", BAD_BOTH + [
    (dict(grad_dtype=BF16), EDTYPE), (dict(dy=None), EINVAL), (dict(dx=None), EINVAL), (dict(lddx=3), EINVAL),
    (dict(mean=None), EINVAL), (dict(rstd=None), EINVAL), (dict(dweight=0x5001), EINVAL),
    (dict(workspace=None), EINVAL), (dict(workspace=0x100008), EINVAL), (dict(workspace_bytes=127), EINVAL),
    (dict(workspace_bytes=-1), EINVAL), (dict(dbias=0x5000), EINVAL), (dict(dweight=0x1000), EINVAL),
    (dict(dx=0x100000), EINVAL), (dict(dh=0x40000, lddh=16), EINVAL), (dict(dresidual=0x50000), EINVAL),
])
def test_norm_backward_refuses(over, code):
    assert L.gclip_layernorm_backward(bwd(**over), None) == code


def test_residual_backward_refuses():
    d = drop()
    assert L.gclip_residual_backward(bwd(**RES_B), None, None) == EINVAL            # dx without dropout
    assert L.gclip_residual_backward(bwd(**RES_B, **{"dx": None}), d, None) == EINVAL   # none with it
    for over in (dict(dresidual=None), dict(dresidual=0x30000), dict(dh=0x40001), dict(lddh=-2)):
        assert L.gclip_residual_backward(bwd(**{**RES_B, **over}), d, None) == EINVAL, over


@pytest.mark.parametrize("d", [drop(-0.1), drop(1.5), drop(float("nan")), drop(d_step=0x1002)])
def test_bad_dropouts_are_refused(d):
    assert L.gclip_dropout_apply(0x1000, 8, 0x2000, 8, 4, 8, F32, d, None) == EINVAL
    assert L.gclip_residual_forward(fwd(**RES_F), d, None) == EINVAL
    assert L.gclip_residual_backward(bwd(**RES_B), d, None) == EINVAL


def test_dropout_refuses():
    d = drop()
    assert L.gclip_dropout_apply(0x1000, 8, 0x2000, 8, 4, 8, F32, None, None) == EINVAL
    assert L.gclip_dropout_apply(0x1000, 8, 0x2000, 8, 4, 8, 7, d, None) == EDTYPE
    for x, ldx, y, ldy, rows, size in ((None, 8, 0x2000, 8, 4, 8), (0x1000, 8, None, 8, 4, 8),
                                       (0x1000, 8, 0x2000, 7, 4, 8), (0x1000, -8, 0x2000, 8, 4, 8),
                                       (0x1000, 8, 0x1010, 8, 4, 8), (0x1000, 8, 0x2000, 8, -4, 8),
                                       (0x1000, 8, 0x2000, 8, 4, -8), (0x1000, 8, 0x2000, 8, MOST + 1, 8)):
        assert L.gclip_dropout_apply(x, ldx, y, ldy, rows, size, F32, d, None) == EINVAL


def test_null_structures_are_refused():
    assert L.gclip_layernorm_forward(None, None) == EINVAL
    assert L.gclip_residual_forward(None, None, None) == EINVAL
    assert L.gclip_layernorm_backward(None, None) == EINVAL
    assert L.gclip_residual_backward(None, None, None) == EINVAL


def test_calls_without_rows_do_nothing():
    none = dict(x=None, y=None, mean=None, rstd=None)
    assert L.gclip_layernorm_forward(fwd(rows=0, **none), None) == OK
    assert L.gclip_residual_forward(fwd(rows=0, **none), drop(), None) == OK
    assert L.gclip_dropout_apply(None, 8, None, 8, 0, 8, F32, drop(), None) == OK
    assert L.gclip_dropout_apply(None, 8, None, 8, 8, 0, F32, drop(), None) == OK
    none = dict(dy=None, x=None, dx=None, mean=None, rstd=None)
    assert L.gclip_layernorm_backward(bwd(rows=0, dweight=None, dbias=None, **none), None) == OK
    assert L.gclip_layernorm_backward(bwd(rows=0, accumulate=1, **none), None) == OK


def test_workspace():
    assert L.gclip_layer_workspace(-1, 8) == 0 and L.gclip_layer_workspace(8, 0) == 0
    for rows in (0, 1, 17, 4096, MOST):
        for size in (1, 7, 768, 16384, 1 << 22, MOST):
            n = L.gclip_layer_workspace(rows, size)
            if rows == 0:
                assert n == 0
            else:
                assert 8 * size <= n <= max(8 * size, 64 << 20) + 8 * rows and n % 8 == 0


def _bytes_of(at, ld, rows, size, es=4):
    return {b for r in range(rows) for b in range(at + r * ld * es, at + r * ld * es + size * es)}


def test_overlaps_against_every_byte():
    """A dropout between two matrices is refused exactly when they share a
    byte and are not the same matrix (equal ld), or may share one (other ld:
    the spans meet)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("valid calls would reach the GPU with these addresses")
    d = drop()
    for rows, size, ld in ((1, 4, 4), (3, 4, 4), (3, 4, 9), (2, 5, 12)):
        base = 0x100000
        for off in range(-30, 31):
            y = base + 4 * off
            got = L.gclip_dropout_apply(base, ld, y, ld, rows, size, F32, d, None)
            share = bool(_bytes_of(base, ld, rows, size) & _bytes_of(y, ld, rows, size))
            assert (got == EINVAL) == (share and off != 0), (rows, size, ld, off, got)
        for off in (-60, -3, 0, 3, 60):
            got = L.gclip_dropout_apply(base, ld + 3, base + 4 * off, ld, rows + 1, size, F32, d, None)
            spans = -(rows * ld + size) < off < rows * (ld + 3) + size
            assert (got == EINVAL) == spans, (rows, size, ld, off, got)


def test_structures_have_the_sizes_of_the_header():
    assert ctypes.sizeof(_lib.GclipDropout) == 32
    assert ctypes.sizeof(_lib.GclipLayerForward) == 17 * 8 - 8
    assert ctypes.sizeof(_lib.GclipLayerBackward) == 23 * 8 - 16


def test_tensors_and_masks_that_no_gpu_sees_are_refused():
    import torch

    import global_l2_norm_amd as G
    x, w = torch.ones(4, 16), torch.ones(16)
    m = G.DropoutMask(0.5, 1, step=3, site=4)
    for call in (lambda: G.layer_norm_forward(x, w), lambda: G.residual_norm_forward(x, x, w),
                 lambda: G.layer_norm_backward(x, x, w[:4], w[:4], w), lambda: G.dropout_forward(x, m),
                 lambda: G.layer_norm(x, w), lambda: G.dropout(x.requires_grad_(), m)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        G.layer_norm_forward(x.double())
    for p, seed, kw in ((-1e-9, 0, {}), (1.0 + 1e-9, 0, {}), (float("nan"), 0, {}), (0.5, -1, {}), (0.5, 1 << 64, {}),
                        (0.5, 0, dict(step=-1)), (0.5, 0, dict(step=1 << 32)), (0.5, 0, dict(site=1 << 32)),
                        (0.5, 0, dict(counter=torch.zeros(1, dtype=torch.int32)))):
        with pytest.raises(ValueError):
            G.DropoutMask(p, seed, **kw)
    other = m.at(site=9)
    assert (other.p, other.seed, other.step, other.site) == (0.5, 1, 3, 9)
    assert G.DropoutMask(2.0 ** -17, 0).drops and not G.DropoutMask(2.0 ** -17 - 1e-9, 0).drops


def test_forward_mode_derivatives_are_refused():
    """A tensor with a tangent has no gradient of its own; without a check the
    result would come back without a tangent, as if it were constant."""
    import torch
    import torch.autograd.forward_ad as forward_ad

    import global_l2_norm_amd as G
    from global_l2_norm_amd import layers
    m = G.DropoutMask(0.5, 1)
    x, w = torch.ones(4, 16), torch.ones(16)
    with forward_ad.dual_level():
        dx, dw = forward_ad.make_dual(x, x), forward_ad.make_dual(w, w)
        for call in (lambda: G.layer_norm(dx, w), lambda: G.layer_norm(x, dw), lambda: G.layer_norm(x, w, dw),
                     lambda: G.dropout(dx, m), lambda: G.residual_norm(dx, x), lambda: G.residual_norm(x, dx, mask=m),
                     lambda: layers._matrix_of(dx)):
            for mode in (torch.enable_grad, torch.no_grad):
                with mode(), pytest.raises(NotImplementedError):
                    call()
        for call in (lambda: G.layer_norm(x, w), lambda: G.dropout(x, m)):
            with pytest.raises(ValueError, match="device"):  # no tangent: only that no GPU sees it
                call()
    for call in (lambda t: G.layer_norm(t, w), lambda t: G.dropout(t, m)):
        with pytest.raises(NotImplementedError):
            torch.func.jvp(call, (x,), (x,))


def test_tracing_is_refused():
    """torch.jit.trace records torch operations, not kernels that a C call
    enqueues: the trace would return memory that nothing wrote."""
    import torch

    import global_l2_norm_amd as G
    m = G.DropoutMask(0.5, 1)
    x, w = torch.ones(4, 16), torch.ones(16)
    grad = x.clone().requires_grad_()
    for call, arg in ((lambda t: G.layer_norm(t, w), x), (lambda t: G.layer_norm(t, w), grad),
                      (lambda t: G.dropout(t, m), x), (lambda t: G.residual_norm(t, x, mask=m)[1], x),
                      (lambda t: G.layer_norm_backward(x, t, w[:4], w[:4], w)[0], x)):
        with pytest.raises(RuntimeError, match="traced"):
            torch.jit.trace(call, arg)


def test_masks_do_not_change():
    """What the kernels take is fixed when a mask is made: a changed attribute
    would be ignored."""
    import copy
    import pickle

    import global_l2_norm_amd as G
    m = G.DropoutMask(0.5, 1, step=3, site=4)
    for name, value in (("p", 0.1), ("seed", 2), ("step", 5), ("site", 6), ("counter", None), ("args", None),
                        ("other", 1)):
        with pytest.raises(AttributeError):
            setattr(m, name, value)
    with pytest.raises(AttributeError):
        m.step += 1
    assert (m.p, m.seed, m.step, m.site, m.args.step, m.args.site) == (0.5, 1, 3, 4, 3, 4)
    assert m.at(step=5).args.step == 5
    for other in (copy.copy(m), copy.deepcopy(m), pickle.loads(pickle.dumps(m))):
        assert bytes(other.args) == bytes(m.args) and other.site == 4


def test_the_profile_summary_is_of_the_present_kernels():
    """profiles/layers__trace_pmc.txt names the code it was taken on, without
    its comments."""
    import hashlib
    import os
    import re

    import bench
    csrc = os.path.join("global_l2_norm_amd", "csrc")
    h = hashlib.sha256()
    for f in sorted(os.listdir(os.path.join(bench.ROOT, csrc))):
        if f.startswith("gclip_layer"):
            with open(os.path.join(bench.ROOT, csrc, f), encoding="utf-8") as src:
                h.update(bench._code_only(src.read()).encode())
    with open(os.path.join(bench.PROFILES, "layers__trace_pmc.txt")) as f:
        assert re.search(r"^kernel_source_sha256_16: (\w+)$", f.read(), re.M)[1] == h.hexdigest()[:16]
