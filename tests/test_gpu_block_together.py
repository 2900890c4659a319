"""The block operators and the log probabilities as they are used together: a
training step by passes, each operator's results held against the oracle at
what it was given, and the served token's products of 8-bit operands."""
import numpy as np
import pytest

from oracle import block as B
from tests import block_util as bu
from tests import layers_util as lu
from tests.test_gpu_block import EPS, G, _need_gpu, bits, mask  # noqa: F401
from tests.test_gpu_layers import factors, stored_sum
from tests.test_gpu_logprob import chain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_training_step_by_passes(dtype, checkpoint):
    """Two microbatches: residual step and norm, the gated product, residual
    step and norm, logits, log probabilities and entropies; back again, the
    norms' weight gradients added up where a GradList clips them."""
    import torch
    g, rng, t = G(), np.random.default_rng(1), lu.torch_type(dtype)
    rows, width, inner, vocabulary = 96, 200, 328, 1003
    new = lambda *s, std=1.0: torch.from_numpy(std * rng.standard_normal(s)).to(t).cuda()  # noqa: E731
    w1, w2 = torch.ones(width, device="cuda"), torch.ones(width, device="cuda")
    into, down = new(width, 2 * inner, std=width ** -0.5), new(inner, width, std=inner ** -0.5)
    head = new(width, vocabulary, std=width ** -0.5)
    grads = [torch.zeros(width, device="cuda") for _ in range(2)] + [torch.zeros(s, device="cuda", dtype=torch.float32) for s in
                                                                     (into.shape, down.shape, head.shape)]
    v = lu.values
    expect = [np.zeros(width), np.zeros(width)]
    for micro in range(2):
        x, stream = new(rows, width), new(rows, width)
        targets = torch.from_numpy(rng.integers(0, vocabulary, rows)).cuda()
        targets[::7] = -100
        m1, m2 = mask(site=2 * micro), mask(site=2 * micro + 1)
        f1, f2 = factors(rows, width, site=2 * micro), factors(rows, width, site=2 * micro + 1)

        h1, y1, r1, k1 = g.residual_rms_norm_forward(x, stream, w1, EPS, m1, keep=checkpoint)
        assert np.array_equal(v(h1), stored_sum(v(stream), v(x), f1, dtype))
        bu.check_rms(v(h1), v(y1), v(r1), v(w1), EPS, dtype, "first norm")
        both = y1 @ into
        z, g8, u8 = g.activation_forward(both[:, :inner], both[:, inner:], keep=checkpoint)
        out = z @ down
        h2, y2, r2, k2 = g.residual_rms_norm_forward(out, h1, w2, EPS, m2, keep=checkpoint)
        assert np.array_equal(v(h2), stored_sum(v(h1), v(out), f2, dtype))
        bu.check_rms(v(h2), v(y2), v(r2), v(w2), EPS, dtype, "second norm")
        logits = y2 @ head
        p = g.token_log_probs_forward(logits, targets, entropy=True)
        m, s, zz, pp, hh = B.log_probs(v(logits))
        ts, tz, th = bu.log_prob_tolerances(v(logits), chain(vocabulary, dtype))
        counted = targets.cpu().numpy() >= 0
        want = zz[np.arange(rows), np.maximum(targets.cpu().numpy(), 0)] * counted
        lu.within(v(p.logp), want, tz + 2 * lu.U * np.abs(want), "logp")
        lu.within(v(p.entropy), hh * counted, th, "entropy")

        dlogp = torch.full((rows,), -1.0 / rows, device="cuda")
        dentropy = torch.full((rows,), -0.01 / rows, device="cuda")
        dlogits = g.token_log_probs_backward(dlogp, dentropy, logits, targets, p.stats, p.entropy)
        wantd = B.log_probs_gradient(v(logits), targets.cpu().numpy(), v(dlogp), v(dentropy), v(p.stats)[:, 0], v(p.stats)[:, 1], v(p.entropy))
        a = np.abs(np.where(np.isfinite(zz), zz, 0))
        tol = pp * (1 / rows + 0.01 / rows * (a + np.abs(v(p.entropy))[:, None])) * (3.5 * a + 2 * np.abs(s)[:, None] + 12) * lu.U
        lu.within(v(dlogits), wantd, bu.stored(wantd, dtype, tol + 3 * lu.U * np.abs(wantd) + 2.0 ** -126), "dlogits")
        grads[4] += (y2.t() @ dlogits).float()
        dy2 = dlogits @ head.t()
        dout, dh1, _ = g.residual_rms_norm_backward(dy2, None, k2 or h2, r2, w2, m2, dweight=grads[1], accumulate=True)
        n2 = bu.packed_values(k2)[2] if checkpoint else v(h2)
        expect[1] = expect[1].astype(np.float32).astype(np.float64)
        bu.check_rms_gradient(v(dout), v(grads[1]), v(dy2), n2, v(r2), v(w2), dtype, "f32", "second norm", None, f2, v(dh1), expect[1])
        expect[1] = v(grads[1])
        dz = dout @ down.t()
        dboth = torch.empty_like(both)
        gate, up = (g8, u8) if checkpoint else (both[:, :inner], both[:, inner:])
        _, _, again = g.activation_backward(dz, gate, up, recompute=True, out_gate=dboth[:, :inner], out_up=dboth[:, inner:])
        a = bu.packed_values(g8)[2] if checkpoint else v(gate)
        b = bu.packed_values(u8)[2] if checkpoint else v(up)
        # the kept values' own product is rounded to binary32 first: u of it
        (wy, ws), (ty, ts) = B.act("silu", a), bu.act_tolerances("silu", a)
        ty, ts = ty + checkpoint * lu.U * np.abs(a) * 1.1, ts + checkpoint * lu.U * np.abs(a) * 0.5
        wg, wu = v(dz) * b * ws, v(dz) * wy
        lu.within(v(dboth[:, :inner]), wg, bu.stored(wg, dtype, np.abs(v(dz) * b) * (ts + 4 * lu.U * np.abs(ws))), "dgate")
        lu.within(v(dboth[:, inner:]), wu, bu.stored(wu, dtype, np.abs(v(dz)) * ty + 2 * lu.U * np.abs(wu)), "dup")
        if not checkpoint:
            assert bits(again) == bits(z)
        grads[3] += (again.t() @ dout).float()
        grads[2] += (y1.t() @ dboth).float()
        dy1 = dboth @ into.t()
        dx, dstream, _ = g.residual_rms_norm_backward(dy1, dh1, k1 or h1, r1, w1, m1, dweight=grads[0], accumulate=True)
        n1 = bu.packed_values(k1)[2] if checkpoint else v(h1)
        bu.check_rms_gradient(v(dx), v(grads[0]), v(dy1), n1, v(r1), v(w1), dtype, "f32", "first norm", v(dh1), f1, v(dstream), expect[0])
        expect[0] = v(grads[0])

    total = np.sqrt(sum((v(t) ** 2).sum() for t in grads) / 4)  # of the mean over the microbatches
    before = [v(t) for t in grads]
    lst = g.GradList(grads)
    lst.clip_(total / 2, avg_factor=0.5)
    status, r = lst.read()
    lst.close()
    assert status == 0 and r["clipped"] and abs(r["norm"] - total) <= 1e-6 * total
    for t, b in zip(grads, before):
        lu.within(v(t), b * 0.25, 2e-6 * np.abs(b) + 2.0 ** -149, "clipped")


def test_a_nan_kept_in_8_bits_stops_the_clip():
    """What is not finite stays so through a checkpoint, up to the list's
    check."""
    import torch
    g = G()
    x = torch.randn(64, 300, device="cuda", dtype=torch.bfloat16)
    x[5, 7] = float("inf")
    w = torch.ones(300, device="cuda").requires_grad_()
    y = g.rms_norm(x, w, EPS, checkpoint=True)
    y.backward(torch.ones_like(y))
    lst = g.GradList([w.grad])
    lst.clip_(1.0, error_if_nonfinite=True)
    status, r = lst.read(error_if_nonfinite=True)
    lst.close()
    assert r["nonfinite"] and r["skipped"]


@pytest.mark.parametrize("rows", [1, 16, 33])
def test_served_tokens_products_of_8_bit_operands(rows):
    """The norm's output with a scale a row as the library's scaled product
    takes it: values, and a column of scales."""
    import torch
    g, rng = G(), np.random.default_rng(2)
    width, n = 512, 256
    x, r = (lu.matrix(rng.standard_normal((rows, width)), "bf16") for _ in range(2))
    w = torch.ones(width, device="cuda", dtype=torch.bfloat16)
    into = g.pack8(torch.from_numpy(rng.standard_normal((n, width))).float().cuda(), "row")
    h, y8, _, _ = g.residual_rms_norm_forward(x, r, w, EPS, packed="row", stats=False)
    bu.check_rms(lu.values(h), y8, None, lu.values(w), EPS, "bf16", "y8", "row")
    out = torch._scaled_mm(y8.values, into.values.t(), scale_a=y8.scales, scale_b=into.scales.t(), out_dtype=torch.bfloat16)
    a, b = bu.packed_values(y8)[2], bu.packed_values(into)[2]
    want = a @ b.T
    tol = (width + 4) * lu.U * (np.abs(a) @ np.abs(b).T)
    lu.within(lu.values(out), want, bu.stored(want, "bf16", tol), "product")


def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_lm.py")
    spec = importlib.util.spec_from_file_location("gated_lm", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("bf16,checkpoint,entropy", [(False, False, 0.0), (True, True, 0.01), (False, True, 0.0)])
def test_the_example_runs(bf16, checkpoint, entropy):
    import torch
    losses, norms = _example().train(3, dtype=torch.bfloat16 if bf16 else torch.float32, checkpoint=checkpoint, entropy=entropy)
    assert len(losses) == len(norms) == 3 and np.isfinite(losses).all() and np.isfinite(norms).all() and min(norms) > 0


def test_the_examples_gradients():
    """Against the model written in binary64 torch operations.  Each of the
    about 25 steps from the embeddings to the loss and back is off by at most
    (K + 10) u of its result's norm, with K <= 512 terms a sum, 25 522 2^-24 =
    8e-4 in all, and errors grow from step to step by what the blocks pass on
    of them, for which a factor of 10 stands."""
    import torch
    e = _example()
    model = e.Model(seed=3)
    generator = torch.Generator().manual_seed(4)
    tokens, targets = e.batch(torch.randperm(257, generator=generator), 4, 16, generator)
    model.loss(tokens, targets, entropy=0.05).backward()

    p = [t.detach().double().cpu().requires_grad_() for t in model.params]
    emb, norms, rest = p[0], p[1:5], p[5:]
    rms = lambda h, w: h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    x = emb[tokens.cpu().reshape(-1)]
    h = torch.zeros_like(x)
    for i in range(3):
        h = h + x
        both = rms(h, norms[i]) @ rest[2 * i]
        gate, up = both[:, :512], both[:, 512:]
        x = (gate * torch.sigmoid(gate) * up) @ rest[2 * i + 1]
    z = torch.log_softmax(rms(h + x, norms[3]) @ emb.t(), 1)
    t = targets.cpu().reshape(-1)
    counted = t != -100
    logp = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    entropy = -(z.exp() * z).sum(1)
    loss = -((logp + 0.05 * entropy) * counted).sum() / counted.sum()
    loss.backward()
    for i, (a, b) in enumerate(zip(model.params, p)):
        off = (a.grad.double().cpu() - b.grad).norm() / b.grad.norm()
        assert off <= 8e-3, (i, float(off))


def test_the_readme_runs():
    """README.md's example of these operators."""
    import os
    import re

    import torch

    import global_l2_norm_amd as g
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        block, = (b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "residual_rms_norm" in b)
    torch.manual_seed(3)
    make = lambda *n: torch.randn(*n, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    env = dict(G=g, x=make(20, 64).requires_grad_(), residual=make(20, 64), weight=make(64), w_gate=make(96, 64),
               w_up=make(96, 64), logits=make(20, 1000).requires_grad_(), targets=torch.arange(20, device="cuda"),
               mask=g.DropoutMask(0.1, 1))
    exec(block, env)
    (env["loss"] + env["r"].entropy.sum() + env["z"].float().sum()).backward()
    assert torch.isfinite(env["x"].grad).all() and torch.isfinite(env["logits"].grad).all()
    assert torch.equal(env["logits"].gather(1, env["best"].top_ids), env["logits"].topk(20, dim=1).values)
    assert env["y8"].values.dtype == torch.float8_e4m3fn and env["y8"].scales.shape == (20, 1)
