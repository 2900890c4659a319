"""The block and log probability calls of the C ABI on the CPU: argument
errors come back before any GPU work.  No call here has valid arguments and
rows at once, but for the ones of the overlap test, which runs only where there
is no GPU to reach."""
import ctypes

import pytest

from global_l2_norm_amd import _lib

L = _lib.lib
OK, EINVAL, EDTYPE = _lib.GCLIP_OK, _lib.GCLIP_EINVAL, _lib.GCLIP_EDTYPE
F32, F16, BF16 = _lib.GCLIP_F32, _lib.GCLIP_F16, _lib.GCLIP_BF16
BLOCK, ROW = _lib.GCLIP_SCALES_BLOCK, _lib.GCLIP_SCALES_ROW
MOST = 0x7ffffff0


def packed(values=None, ld=16, scales=None, mode=BLOCK, reserved=0):
    return _lib.GclipPacked8(values, ld, scales, mode, reserved)


def fwd(**over):
    a = dict(rows=4, size=16, dtype=F32, weight_dtype=F32, eps=1e-5, x=0x10000, ldx=16, residual=None, ldresidual=0,
             weight=0x1000, h=None, ldh=0, y=0x20000, ldy=16, y8=packed(), kept=packed(), rstd=0x4000)
    a.update(over)
    return _lib.GclipRmsForward(**a)


def bwd(**over):
    a = dict(rows=4, size=16, dtype=F32, weight_dtype=F32, grad_dtype=F32, accumulate=0, dy=0x10000, lddy=16, dh=None,
             lddh=0, x=0x20000, ldx=16, x8=packed(), rstd=0x4000, weight=0x1000, dresidual=None, lddresidual=0,
             dx=0x30000, lddx=16, dweight=0x5000, workspace=0x100000, workspace_bytes=1 << 20)
    a.update(over)
    return _lib.GclipRmsBackward(**a)


def act(**over):
    a = dict(rows=4, size=16, dtype=F32, kind=0, gate=0x10000, ldgate=16, up=0x20000, ldup=16, gate8=packed(),
             up8=packed(), y=0x30000, ldy=16, dy=None, lddy=0, dgate=None, lddgate=0, dup=None, lddup=0)
    a.update(over)
    return _lib.GclipActivate(**a)


ACT_B = dict(dy=0x40000, lddy=16, dgate=0x50000, lddgate=16, dup=0x60000, lddup=16, y=None)


def logp(**over):
    a = dict(rows=4, size=16, dtype=F32, top=0, logits=0x10000, ld=16, targets=0x1000, ignore=-100, stats=0x2000,
             logp=0x3000, entropy=0x4000, top_logp=None, top_ids=None, dlogp=None, dentropy=None, dlogits=None,
             lddlogits=0, workspace=0x100000, workspace_bytes=1 << 20)
    a.update(over)
    return _lib.GclipLogprobs(**a)


LOGP_B = dict(logp=None, dlogp=0x5000, dentropy=0x6000, dlogits=0x20000, lddlogits=16)
RES_F = dict(residual=0x30000, ldresidual=16, h=0x40000, ldh=16)
RES_B = dict(dh=0x40000, lddh=16, dresidual=0x50000, lddresidual=16)


def drop(p=0.5, **over):
    a = dict(p=p, seed=1, step=0, site=0, d_step=None)
    a.update(over)
    return _lib.GclipDropout(**a)


EXTENTS = [(dict(rows=-1), EINVAL), (dict(rows=MOST + 1), EINVAL), (dict(size=0), EINVAL), (dict(size=-3), EINVAL),
           (dict(size=MOST + 1), EINVAL), (dict(dtype=3), EDTYPE), (dict(dtype=-1), EDTYPE)]
BAD8 = [packed(0x70000, 16, None), packed(0x70004, 16, 0x8000), packed(0x70000, 12, 0x8000),
        packed(0x70000, 8, 0x8000), packed(0x70000, -16, 0x8000), packed(0x70000, 16, 0x8002),
        packed(0x70000, 16, 0x8000, 2), packed(0x70000, 16, 0x8000, -1), packed(0x70000, 16, 0x8000, BLOCK, 1),
        packed(None, 16, 0x8000)]


class _ByReference:
    """The calls with a structure by reference."""

    def __getattr__(self, name):
        f = getattr(_lib.lib, name)
        return lambda *a: f(*(ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in a))


L = _ByReference()


@pytest.mark.parametrize("over,code", EXTENTS + [
    (dict(weight_dtype=F16), EDTYPE), (dict(dtype=BF16, weight_dtype=F16), EDTYPE), (dict(x=None), EINVAL),
    (dict(x=0x10002), EINVAL), (dict(ldx=-16), EINVAL), (dict(ldx=1 << 60), EINVAL), (dict(weight=0x1001), EINVAL),
    (dict(eps=0.0), EINVAL), (dict(eps=-1e-5), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(eps=float("inf")), EINVAL), (dict(eps=1e39), EINVAL), (dict(eps=1e-39), EINVAL),
    (dict(y=None), EINVAL), (dict(y=0x20001), EINVAL), (dict(ldy=15), EINVAL), (dict(ldy=0), EINVAL),
    (dict(rstd=0x4002), EINVAL), (dict(residual=0x30000), EINVAL), (dict(h=0x40000), EINVAL),
    (dict(y=0x10040), EINVAL),                       # y a row behind x
    (dict(ldx=0, y=0x10000), EINVAL),                # over a broadcast row
    (dict(rstd=0x20010), EINVAL),                    # rstd inside y
    (dict(y8=packed(0x70000, 16, 0x8000)), EINVAL),  # y and y8
    (dict(y=None, y8=packed(0x10000, 16, 0x8000)), EINVAL),   # y8 over x, which no element fits
    (dict(kept=packed(0x70000, 16, 0x8000, ROW)), EINVAL),    # checkpoints have scales by block
    (dict(kept=packed(0x70000, 16, 0x70010)), EINVAL),        # scales among the values
    (dict(kept=packed(0x1000, 16, 0x8000)), EINVAL),          # kept over weight
])
def test_norm_forward_refuses(over, code):
    assert L.gclip_rmsnorm_forward(fwd(**over), None) == code


@pytest.mark.parametrize("bad", BAD8)
def test_bad_matrices_in_8_bits_are_refused(bad):
    if bad.values is not None:  # no values: y is written instead
        assert L.gclip_rmsnorm_forward(fwd(y=None, y8=bad), None) == EINVAL
        assert L.gclip_rmsnorm_backward(bwd(x=None, x8=bad), None) == EINVAL
    assert L.gclip_rmsnorm_forward(fwd(kept=bad), None) == EINVAL
    assert L.gclip_activation_forward(act(up=None, gate8=bad), None) == EINVAL
    assert L.gclip_activation_backward(act(**{**ACT_B, "gate": None, "up": None, "dup": None}, gate8=bad), None) == EINVAL
    assert L.gclip_pack(0x10000, 16, bad, 4, 16, F32, None) == EINVAL
    assert L.gclip_unpack(bad, 0x10000, 16, 4, 16, F32, None) == EINVAL


@pytest.mark.parametrize("over", [
    dict(residual=None), dict(h=None), dict(ldh=8), dict(ldresidual=-1), dict(h=0x20000), dict(h=0x30010),
    dict(kept=packed(0x40000, 16, 0x8000))])
def test_residual_forward_refuses(over):
    assert L.gclip_residual_rms_forward(fwd(**{**RES_F, **over}), None, None) == EINVAL


@pytest.mark.parametrize("over,code", EXTENTS + [
    (dict(grad_dtype=BF16), EDTYPE), (dict(weight_dtype=BF16), EDTYPE), (dict(dy=None), EINVAL),
    (dict(dx=None), EINVAL), (dict(lddx=3), EINVAL), (dict(rstd=None), EINVAL), (dict(dweight=0x5001), EINVAL),
    (dict(rows=4096, workspace=None), EINVAL), (dict(rows=4096, workspace=0x100008), EINVAL),
    (dict(rows=4096, workspace_bytes=63), EINVAL), (dict(workspace_bytes=-1), EINVAL), (dict(dweight=0x1000), EINVAL),
    (dict(rows=4096, dy=0x1000000, x=0x2000000, dx=0x100000, workspace_bytes=1 << 24), EINVAL),
    (dict(dh=0x40000, lddh=16), EINVAL), (dict(dresidual=0x50000), EINVAL), (dict(x=None), EINVAL),
    (dict(x8=packed(0x70000, 16, 0x8000)), EINVAL),                   # x and x8
    (dict(x=None, x8=packed(0x30000, 16, 0x8000)), EINVAL),           # x8 under dx
    (dict(x=None, x8=packed(0x70000, 16, 0x30000)), EINVAL),          # its scales too
])
def test_norm_backward_refuses(over, code):
    assert L.gclip_rmsnorm_backward(bwd(**over), None) == code


def test_residual_backward_refuses():
    d = drop()
    assert L.gclip_residual_rms_backward(bwd(**RES_B), None, None) == EINVAL               # dx without dropout
    assert L.gclip_residual_rms_backward(bwd(**RES_B, **{"dx": None}), d, None) == EINVAL  # none with it
    for over in (dict(dresidual=None), dict(dresidual=0x30000), dict(dh=0x40001), dict(lddh=-2)):
        assert L.gclip_residual_rms_backward(bwd(**{**RES_B, **over}), d, None) == EINVAL, over


@pytest.mark.parametrize("d", [drop(-0.1), drop(1.5), drop(float("nan")), drop(d_step=0x1002)])
def test_bad_dropouts_are_refused(d):
    assert L.gclip_residual_rms_forward(fwd(**RES_F), d, None) == EINVAL
    assert L.gclip_residual_rms_backward(bwd(**RES_B), d, None) == EINVAL


@pytest.mark.parametrize("over,code", EXTENTS + [
    (dict(kind=-1), EINVAL), (dict(kind=4), EINVAL), (dict(gate=None), EINVAL), (dict(y=None), EINVAL),
    (dict(ldgate=-1), EINVAL), (dict(ldy=3), EINVAL), (dict(up=0x20001), EINVAL),
    (dict(gate8=packed(0x70000, 16, 0x8000)), EINVAL),                                   # up8 is missing
    (dict(up8=packed(0x70000, 16, 0x8000)), EINVAL),                                     # gate8 is
    (dict(up=None, gate8=packed(0x70000, 16, 0x8000), up8=packed(0x90000, 16, 0x9000)), EINVAL),  # up is
    (dict(gate8=packed(0x70000, 16, 0x8000, ROW), up8=packed(0x90000, 16, 0x9000)), EINVAL),
    (dict(gate8=packed(0x70000, 16, 0x8000), up8=packed(0x70000, 16, 0x9000)), EINVAL),
    (dict(dy=0x40000), EINVAL), (dict(dgate=0x50000), EINVAL), (dict(dup=0x50000), EINVAL),
    (dict(y=0x10004), EINVAL),
])
def test_activation_forward_refuses(over, code):
    assert L.gclip_activation_forward(act(**over), None) == code


@pytest.mark.parametrize("over,code", EXTENTS + [
    (dict(kind=9), EINVAL), (dict(dy=None), EINVAL), (dict(dgate=None), EINVAL), (dict(dup=None), EINVAL),
    (dict(up=None), EINVAL),                               # dup without up
    (dict(gate=None), EINVAL), (dict(lddup=2), EINVAL), (dict(dup=0x50000), EINVAL), (dict(y=0x50000, ldy=16), EINVAL),
    (dict(gate8=packed(0x70000, 16, 0x8000), up8=packed(0x90000, 16, 0x9000)), EINVAL),  # gate too
    (dict(gate=None, gate8=packed(0x70000, 16, 0x8000), up8=packed(0x90000, 16, 0x9000)), EINVAL),  # up too
    (dict(gate=None, up=None, gate8=packed(0x70000, 16, 0x8000)), EINVAL),               # dup without up8
])
def test_activation_backward_refuses(over, code):
    assert L.gclip_activation_backward(act(**{**ACT_B, **over}), None) == code


def test_pack_refuses():
    p = packed(0x70000, 16, 0x8000)
    assert L.gclip_pack(0x10000, 16, None, 4, 16, F32, None) == EINVAL
    assert L.gclip_unpack(None, 0x10000, 16, 4, 16, F32, None) == EINVAL
    assert L.gclip_pack(0x10000, 16, p, 4, 16, 5, None) == EDTYPE
    assert L.gclip_unpack(p, 0x10000, 16, 4, 16, 5, None) == EDTYPE
    for x, ld, rows, size in ((None, 16, 4, 16), (0x10001, 16, 4, 16), (0x10000, -1, 4, 16), (0x10000, 16, -1, 16),
                              (0x10000, 16, 4, 0), (0x10000, 16, MOST + 1, 16), (0x6fff0, 16, 4, 16)):
        assert L.gclip_pack(x, ld, p, rows, size, F32, None) == EINVAL, (x, ld, rows, size)
        assert L.gclip_unpack(p, x, ld, rows, size, F32, None) == EINVAL, (x, ld, rows, size)
    assert L.gclip_unpack(p, 0x10000, 15, 4, 16, F32, None) == EINVAL
    assert L.gclip_pack(0x10000, 16, packed(), 4, 16, F32, None) == EINVAL
    assert L.gclip_unpack(packed(), 0x10000, 16, 4, 16, F32, None) == EINVAL


@pytest.mark.parametrize("over,code", EXTENTS + [
    (dict(logits=None), EINVAL), (dict(logits=0x10002), EINVAL), (dict(ld=-1), EINVAL), (dict(top=-1), EINVAL),
    (dict(top=33, size=64, ld=64), EINVAL), (dict(top=17), EINVAL), (dict(top=2), EINVAL),
    (dict(top=2, top_logp=0x7000), EINVAL), (dict(top=2, top_ids=0x7000), EINVAL),
    (dict(top_logp=0x7000, top_ids=0x8000), EINVAL), (dict(targets=None), EINVAL), (dict(logp=None), EINVAL),
    (dict(targets=0x1004), EINVAL), (dict(stats=0x2001), EINVAL), (dict(stats=0x2ff8), EINVAL), (dict(logp=0x10000), EINVAL),
    (dict(dlogp=0x5000), EINVAL), (dict(dentropy=0x5000), EINVAL), (dict(dlogits=0x20000), EINVAL),
    (dict(size=100000, ld=100000, workspace=None), EINVAL), (dict(size=100000, ld=100000, workspace_bytes=64), EINVAL),
    (dict(size=100000, ld=100000, workspace=0x100008), EINVAL),
])
def test_log_probs_forward_refuses(over, code):
    assert L.gclip_logprob_forward(logp(**over), None) == code


@pytest.mark.parametrize("over,code", EXTENTS + [
    (dict(logits=None), EINVAL), (dict(dlogits=None), EINVAL), (dict(lddlogits=15), EINVAL), (dict(targets=None), EINVAL),
    (dict(stats=None), EINVAL), (dict(dlogp=None), EINVAL), (dict(entropy=None), EINVAL), (dict(top=1), EINVAL),
    (dict(logp=0x3000), EINVAL), (dict(top_ids=0x3000), EINVAL), (dict(dlogits=0x10020), EINVAL),
    (dict(dlogits=0x2000 - 8), EINVAL),
])
def test_log_probs_backward_refuses(over, code):
    assert L.gclip_logprob_backward(logp(**{**LOGP_B, **over}), None) == code


def test_null_structures_are_refused():
    for f in (L.gclip_rmsnorm_forward, L.gclip_rmsnorm_backward, L.gclip_activation_forward,
              L.gclip_activation_backward, L.gclip_logprob_forward, L.gclip_logprob_backward):
        assert f(None, None) == EINVAL
    assert L.gclip_residual_rms_forward(None, None, None) == EINVAL
    assert L.gclip_residual_rms_backward(None, None, None) == EINVAL


def test_calls_without_rows_do_nothing():
    none = dict(x=None, y=None, rstd=None)
    assert L.gclip_rmsnorm_forward(fwd(rows=0, **none), None) == OK
    assert L.gclip_residual_rms_forward(fwd(rows=0, **none), drop(), None) == OK
    none = dict(dy=None, x=None, dx=None, rstd=None)
    assert L.gclip_rmsnorm_backward(bwd(rows=0, dweight=None, **none), None) == OK
    assert L.gclip_rmsnorm_backward(bwd(rows=0, accumulate=1, **none), None) == OK
    assert L.gclip_activation_forward(act(rows=0, gate=None, up=None, y=None), None) == OK
    assert L.gclip_activation_backward(act(**{**ACT_B, "rows": 0, "up": None, "dup": None}), None) == OK
    assert L.gclip_pack(None, 16, packed(), 0, 16, F32, None) == OK
    assert L.gclip_unpack(packed(), None, 16, 0, 16, F32, None) == OK
    assert L.gclip_logprob_forward(logp(rows=0, logits=None, targets=None), None) == OK
    assert L.gclip_logprob_backward(logp(**{**LOGP_B, "rows": 0}), None) == OK


def test_workspaces():
    assert L.gclip_rms_workspace(-1, 8) == 0 and L.gclip_rms_workspace(8, 0) == 0
    assert L.gclip_rms_workspace(512, 4096) == 0 < L.gclip_rms_workspace(513, 4096) and L.gclip_rms_workspace(512, 4097) > 0
    for rows in (0, 1, 17, 256, 4096, MOST):
        for size in (1, 7, 768, 16384, 1 << 22, MOST):
            n = L.gclip_rms_workspace(rows, size)
            if rows == 0 or (rows <= 256 and 8 <= size <= 16384):  # few rows in registers leave no parts
                assert n == 0
            else:
                assert 4 * size <= n <= max(4 * size, 32 << 20) + 4 * rows
    for bad in ((-1, 8, 0), (8, 0, 0), (8, 8, -1), (8, 8, 9), (8, 64, 33)):
        assert L.gclip_logprob_workspace(*bad) == 0
    for rows in (0, 1, 8, 511, 512, 513, 8192, MOST):
        for size in (1, 64, 1024, 2048, 50304, 1 << 20, MOST):
            for top in (0, min(20, size)):
                n = L.gclip_logprob_workspace(rows, size, top)
                assert 0 <= n <= 512 * 64 * (8 * top + 16) and (n == 0 or rows <= 256)


def test_the_profile_summary_is_of_the_present_kernels():
    """profiles/block__trace_pmc.txt names the code it was taken on, without
    its comments."""
    import hashlib
    import os
    import re

    import bench
    csrc = os.path.join(bench.ROOT, "global_l2_norm_amd", "csrc")
    h = hashlib.sha256()
    for f in sorted(os.listdir(csrc)):
        if re.match("gclip_(block|rms|activation|pack8|operand|logprob)", f):
            with open(os.path.join(csrc, f), encoding="utf-8") as src:
                h.update(bench._code_only(src.read()).encode())
    with open(os.path.join(bench.PROFILES, "block__trace_pmc.txt")) as f:
        assert re.search(r"^kernel_source_sha256_16: (\w+)$", f.read(), re.M)[1] == h.hexdigest()[:16]


def test_overlaps_of_8_bit_rows_against_every_byte():
    """unpack between values and a matrix: refused when any byte is shared,
    those behind a row's end up to a multiple of eight among the values', or
    may be (other distances: the spans meet)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("valid calls would reach the GPU with these addresses")
    base = 0x100000
    for rows, size, ld8, ld in ((1, 4, 8, 4), (3, 13, 16, 4 * 4), (2, 8, 32, 8), (2, 9, 40, 10)):
        whole = (size + 7) // 8 * 8
        for off in range(-48, 49):
            to = base + 4 * off
            got = L.gclip_unpack(packed(base, ld8, 0x8000), to, ld if ld >= size else size, rows, size, F32, None)
            step = (ld if ld >= size else size) * 4
            a = {b for r in range(rows) for b in range(base + r * ld8, base + r * ld8 + whole)}
            c = {b for r in range(rows) for b in range(to + r * step, to + r * step + 4 * size)}
            if step == ld8 or rows == 1:
                assert (got == EINVAL) == bool(a & c), (rows, size, off, got)
            else:
                meet = max(min(a), min(c)) <= min(max(a), max(c))
                assert (got == EINVAL) == meet, (rows, size, off, got)


def test_structures_have_the_sizes_of_the_headers():
    assert ctypes.sizeof(_lib.GclipPacked8) == 32
    assert ctypes.sizeof(_lib.GclipRmsForward) == 14 * 8 + 64
    assert ctypes.sizeof(_lib.GclipRmsBackward) == 20 * 8 - 8 + 32
    assert ctypes.sizeof(_lib.GclipActivate) == 15 * 8 + 64
    assert ctypes.sizeof(_lib.GclipLogprobs) == 18 * 8


def test_tensors_that_no_gpu_sees_are_refused():
    import torch

    import global_l2_norm_amd as G
    x, w, r, t = torch.ones(4, 16), torch.ones(16), torch.ones(4), torch.zeros(4, dtype=torch.int64)
    p = G.Packed8(torch.zeros(4, 16, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(4, 1))
    for call in (lambda: G.rms_norm_forward(x, w), lambda: G.rms_norm(x, w), lambda: G.residual_rms_norm(x, x, w),
                 lambda: G.rms_norm_backward(x, x, r, w), lambda: G.rms_norm_backward(x, p, r, w),
                 lambda: G.activation_forward(x, x), lambda: G.activation(x.clone().requires_grad_()),
                 lambda: G.activation_backward(x, x, x), lambda: G.pack8(x), lambda: p.dequantize(),
                 lambda: G.token_log_probs_forward(x, t), lambda: G.token_log_probs(x, t),
                 lambda: G.token_log_probs_backward(r, None, x, t, torch.ones(4, 2))):
        with pytest.raises(ValueError, match="device"):
            call()
    for call in (lambda: G.rms_norm_forward(x.double()), lambda: G.activation_forward(x.long()),
                 lambda: G.pack8(x.double()), lambda: G.unpack8(x), lambda: G.token_log_probs_forward(x.double(), t)):
        with pytest.raises(TypeError):
            call()


def test_packed_matrices_check_their_layout():
    import torch

    import global_l2_norm_amd as G
    new = lambda *s: torch.zeros(*s, dtype=torch.uint8).view(torch.float8_e4m3fn)  # noqa: E731
    one = torch.ones
    assert G.Packed8(new(4, 256), one(4, 2)).args.mode == BLOCK
    assert G.Packed8(new(4, 256), one(4, 1)).args.mode == ROW
    assert G.Packed8(new(4, 128), one(4, 1)).args.mode == BLOCK  # the same
    assert G.Packed8(new(2, 3, 64), one(2, 3, 1)).args.ld == 64
    assert G.Packed8(new(4, 264)[:, :257], one(4, 3)).args.ld == 264
    assert G.Packed8(new(4, 264)[:, 8:], one(4, 2)).args.ld == 264
    assert G.Packed8(new(0, 257), one(0, 3)).shape == (0, 257)
    for values, scales in ((new(4, 257), one(4, 3)),              # rows at odd addresses
                           (new(4 * 256 + 5)[:1025].view(1, 1025), one(1, 9)),  # no bytes behind the last row
                           (new(4, 264)[:, 4:260], one(4, 2)), (new(256, 4).t(), one(4, 2)),
                           (new(4, 256), one(4, 3)), (new(4, 256), one(3, 2)), (new(4, 256), one(2, 4).t()),
                           (new(4, 3, 8)[:, :2], one(4, 2, 1))):
        with pytest.raises(ValueError):
            G.Packed8(values, scales)
    for values, scales in ((one(4, 256), one(4, 2)), (new(4, 256), one(4, 2).half())):
        with pytest.raises(TypeError):
            G.Packed8(values, scales)
    with pytest.raises(ValueError):
        G.pack8(one(4, 8), "column")


def test_structures_as_bytes():
    """The bytes that the tensors' functions pass are the structure's."""
    a = fwd(y=None, y8=packed(0x70000, 32, 0x8000, ROW), kept=packed(0x90000, 16, 0x9000), **RES_F)
    assert bytes(a) == _lib.PACK_RMS_FORWARD.pack(4, 16, F32, F32, 1e-5, 0x10000, 16, 0x30000, 16, 0x1000, 0x40000, 16, 0, 16,
                                                  0x70000, 32, 0x8000, ROW, 0, 0x90000, 16, 0x9000, BLOCK, 0, 0x4000)
    a = bwd(dtype=BF16, grad_dtype=BF16, accumulate=1, x=None, ldx=3, x8=packed(0x70000, 32, 0x8000), **RES_B)
    assert bytes(a) == _lib.PACK_RMS_BACKWARD.pack(4, 16, BF16, F32, BF16, 1, 0x10000, 16, 0x40000, 16, 0, 3, 0x70000, 32, 0x8000,
                                                   BLOCK, 0, 0x4000, 0x1000, 0x50000, 16, 0x30000, 16, 0x5000, 0x100000, 1 << 20)
    a = act(**{**ACT_B, "kind": 2}, gate8=packed(1, 2, 3), up8=packed(4, 5, 6))
    assert bytes(a) == _lib.PACK_ACTIVATE.pack(4, 16, F32, 2, 0x10000, 16, 0x20000, 16, 1, 2, 3, 0, 0, 4, 5, 6, 0, 0, 0, 16, 0x40000,
                                               16, 0x50000, 16, 0x60000, 16)
    a = logp(top=3, top_logp=1, top_ids=2, dlogp=3, dentropy=4, dlogits=5, lddlogits=6)
    assert bytes(a) == _lib.PACK_LOGPROBS.pack(4, 16, F32, 3, 0x10000, 16, 0x1000, -100, 0x2000, 0x3000, 0x4000, 1, 2, 3, 4, 5, 6,
                                               0x100000, 1 << 20)
    assert _lib.lib.gclip_rmsnorm_forward(bytes(fwd(size=0)), None) == EINVAL


def test_packed_matrices_are_copied():
    import copy

    import torch

    import global_l2_norm_amd as G
    held = torch.arange(4 * 136, dtype=torch.uint8).view(4, 136).view(torch.float8_e4m3fn)
    p = G.Packed8(held[:, :131], torch.rand(4, 2))
    for q in (copy.copy(p), copy.deepcopy(p)):
        assert torch.equal(q.values.view(torch.uint8), p.values.view(torch.uint8)) and torch.equal(q.scales, p.scales)
        assert q.args.ld == 136 and q.args.values == q.values.data_ptr()


def test_forward_mode_derivatives_and_traces_are_refused():
    import torch
    import torch.autograd.forward_ad as forward_ad

    import global_l2_norm_amd as G
    x, w, t = torch.ones(4, 16), torch.ones(16), torch.zeros(4, dtype=torch.int64)
    calls = (lambda v: G.rms_norm(v, w), lambda v: G.residual_rms_norm(x, v, w)[1], lambda v: G.activation(v, x),
             lambda v: G.activation(x, v), lambda v: G.token_log_probs(v, t).logp)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, x)
        for call in calls:
            with pytest.raises(NotImplementedError):
                call(dual)
    for call in calls:
        for arg in (x, x.clone().requires_grad_()):
            with pytest.raises(RuntimeError, match="traced"):
                torch.jit.trace(call, arg)
