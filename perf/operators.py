"""What is measured of the layer operators: layer norm, dropout from a counter-based generator, and the residual step
of a pre-norm block that runs both in one pass (h = residual + dropout(x), y = norm(h)), forward and backward.

With ``own`` false, ``run`` computes them in elementary torch operations; with ``own`` true it makes the calls of
``global_l2_norm_amd``.  The formulas, over the rows of a matrix of `size` columns:

  norm           mean = sum(x) / size, rstd = 1 / sqrt(sum((x - mean)^2) / size + eps), y = (x - mean) rstd w + b
  its gradient   n = (x - mean) rstd, g = dy w, dx = rstd (g - sum(g) / size - n sum(g n) / size),
                 dw = sum over rows of dy n, db = sum over rows of dy (added to what is there when accumulating)
  dropout        y = x s where kept, else 0.  Element (r, c) takes the 16-bit half number c mod 8 (low halves first) of
                 Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011)
                 on the counter (c div 8, r, site, step) under the key (seed's low word, high word), and is kept when
                 that is t = floor(65536 p + 1/2) or more; s = 65536 / (65536 - t).  Its gradient is the same map.
  residual step  h = residual + dropout(x), rounded to its type; y = norm(h).  Its gradient: dresidual = dh + the
                 norm's dx at h, dx = dropout(dresidual).
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OPS = ("norm_forward", "norm_backward", "dropout_forward", "dropout_backward", "residual_forward",
       "residual_backward", "residual_step")


def _case(name, op, rows, size, dtype, weights="f32", p=0.0, stats=True, pad=0, accumulate=False):
    """weights: type of weight, bias and their gradients; stats: keep mean and rstd for a backward pass; pad: columns
    between the end of a row and the next (the inputs are views of a wider buffer)."""
    c = {"op": op, "rows": rows, "size": size, "dtype": dtype, "weights": weights, "p": p, "stats": stats, "pad": pad,
         "accumulate": accumulate}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the final norm of one generated token
        _case("token norm", "norm_forward", 1, 2048, "bf16", "bf16", stats=False),
        # a block's residual add and norm while 32 requests generate one token each: no dropout, nothing kept
        _case("32 tokens residual", "residual_forward", 32, 2048, "f16", "f16", stats=False),
        # a microbatch of 8 sequences of 1024 tokens of the 120M-parameter model that the gradient lists are shaped after
        _case("120M norm", "norm_forward", 8192, 768, "f32"),
        # its backward pass, with the weights' gradients added to those of the microbatches before it
        _case("120M norm gradient", "norm_backward", 8192, 768, "f32", accumulate=True),
        # dropout after its embeddings
        _case("120M dropout", "dropout_forward", 8192, 768, "f32", p=0.1),
        # a microbatch of 16 sequences of 1024 tokens of the 1.3B-parameter bf16 model, binary32 weights
        _case("1.3B norm", "norm_forward", 16384, 2048, "bf16"),
        _case("1.3B norm gradient", "norm_backward", 16384, 2048, "bf16"),
        _case("1.3B dropout gradient", "dropout_backward", 16384, 2048, "bf16", p=0.1),
        # the step between two of its sublayers, each direction
        _case("1.3B residual", "residual_forward", 16384, 2048, "bf16", p=0.1),
        _case("1.3B residual gradient", "residual_backward", 16384, 2048, "bf16", p=0.1),
        # a ragged batch of packed sequences, odd width, inputs that are slices of a wider buffer; both directions
        _case("ragged residual step", "residual_step", 1021, 1111, "f16", p=0.25, pad=5),
        # norms over each attention head's 64 channels
        _case("head norm gradient", "norm_backward", 131071, 64, "bf16", "bf16"),
    ]


def draw(rng):
    op = rng.choice(OPS)
    size = int(round(math.exp(rng.uniform(math.log(32), math.log(16384)))))
    if rng.random() < 0.5:
        size = max(8, size // 64 * 64)
    most = 16384 * 2048 // size // (2 if op == "residual_step" else 1)
    rows = int(round(math.exp(rng.uniform(0.0, math.log(min(most, 131072))))))
    dtype = rng.choice(("f32", "f16", "bf16", "bf16"))
    if dtype == "f32":
        rows = max(1, rows // 2)
    p = 0.0 if op.startswith("norm") or (op.startswith("residual") and rng.random() < 0.25) else rng.choice((0.05, 0.1, 0.3, 0.5))
    stats = op not in ("norm_forward", "residual_forward") or rng.random() < 0.6
    return _case("", op, rows, size, dtype, rng.choice(("f32", dtype)), p, stats, rng.choice((0, 0, 1, 8)),
                 op in ("norm_backward", "residual_backward") and rng.random() < 0.5)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, size, dt, wt = case["rows"], case["size"], DTYPES[case["dtype"]], DTYPES[case["weights"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def matrix(scale=1.0, spread=None, shift=None):
        m = normal(rows, size + case["pad"]).mul_(scale)[:, :size]
        if spread is not None:
            m.mul_(spread).add_(shift)
        return m.to(dt) if case["pad"] == 0 else torch.empty(rows, size + case["pad"], dtype=dt, device="cuda")[:, :size].copy_(m)

    # activations: channels of different spread and offset, a few of them large, as a residual stream has
    spread = 0.5 + torch.rand(size, generator=g, device="cuda")
    spread[torch.randint(0, size, (max(1, size // 256),), generator=g, device="cuda")] *= 8.0
    shift = 0.3 * normal(size)
    s = {"case": case, "seed": (seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 64), "step": seed % 100003, "site": size % 97,
         "p": case["p"], "weight": (1.0 + 0.1 * normal(size)).to(wt), "bias": (0.1 * normal(size)).to(wt)}
    op = case["op"]
    if op in ("norm_forward", "dropout_forward"):
        s["x"] = matrix(1.0, spread, shift)
    elif op == "dropout_backward":
        s["dy"] = matrix(1e-2)
    elif op == "residual_forward":
        s["x"], s["residual"] = matrix(0.5), matrix(1.0, spread, shift)
    elif op == "residual_step":
        s["x"], s["residual"] = matrix(0.5), matrix(1.0, spread, shift)
        s["dy"], s["dh"] = matrix(1e-2), matrix(1e-2)
    else:
        s["h"], s["dy"] = matrix(1.0, spread, shift), matrix(1e-2)
        if op == "residual_backward":
            s["dh"] = matrix(1e-2)
        s["mean"], s["rstd"] = _statistics(s["h"].float())
    if case["accumulate"]:
        s["dweight"], s["dbias"] = (normal(size).mul_(0.1).to(wt) for _ in range(2))
    return s


# ---------------------------------------------------------------- the plain forms
def _statistics(x):
    mean = x.sum(1) / x.shape[1]
    var = (x - mean[:, None]).square().sum(1) / x.shape[1]
    return mean, 1.0 / torch.sqrt(var + EPS)


def _threshold(p):
    return math.floor(65536 * p + 0.5)


def _kept(s, rows, size, device):
    """Truth values [rows, size]: 32-bit words held in int64, whose products wrap to the right 64 bits."""
    low = 0xFFFFFFFF
    groups = (size + 7) // 8
    c0 = torch.arange(groups, device=device).expand(rows, groups)
    c1 = torch.arange(rows, device=device)[:, None].expand(rows, groups)
    c2 = torch.full_like(c0, s["site"])
    c3 = torch.full_like(c0, s["step"])
    k0, k1 = s["seed"] & low, s["seed"] >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & low) ^ c1 ^ k0, b & low, (a >> 32 & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    halves = torch.stack((c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16), -1)
    return halves.reshape(rows, groups * 8)[:, :size] >= _threshold(s["p"])


def _dropout(s, x):
    if s["p"] == 0.0:
        return x
    t = _threshold(s["p"])
    return torch.where(_kept(s, x.shape[0], x.shape[1], x.device), x * (65536.0 / (65536 - t)), torch.zeros_like(x))


def _norm_forward(s, h, dt):
    mean, rstd = _statistics(h)
    y = ((h - mean[:, None]) * rstd[:, None] * s["weight"].float() + s["bias"].float()).to(dt)
    return (y, mean, rstd) if s["case"]["stats"] else (y,)


def _norm_backward(s, dy, h, mean, rstd):
    """dx in binary32 and the weights' gradients."""
    n = (h - mean[:, None]) * rstd[:, None]
    g = dy * s["weight"].float()
    size = h.shape[1]
    dx = rstd[:, None] * (g - g.sum(1, keepdim=True) / size - n * ((g * n).sum(1, keepdim=True) / size))
    dw, db = (dy * n).sum(0), dy.sum(0)
    if s["case"]["accumulate"]:
        dw, db = s["dweight"].copy_(s["dweight"].float() + dw), s["dbias"].copy_(s["dbias"].float() + db)
    return dx, dw.to(s["weight"].dtype), db.to(s["weight"].dtype)


def _plain(s):
    op, dt = s["case"]["op"], DTYPES[s["case"]["dtype"]]
    if op == "norm_forward":
        return _norm_forward(s, s["x"].float(), dt)
    if op == "norm_backward":
        dx, dw, db = _norm_backward(s, s["dy"].float(), s["h"].float(), s["mean"], s["rstd"])
        return dx.to(dt), dw, db
    if op.startswith("dropout"):
        return _dropout(s, s["x" if op == "dropout_forward" else "dy"].float()).to(dt)
    out = ()
    h, stats = s.get("h"), (s.get("mean"), s.get("rstd"))
    if op != "residual_backward":
        h = (s["residual"].float() + _dropout(s, s["x"].float())).to(dt)
        y = _norm_forward(s, h.float(), dt)
        out, stats = (h, *y), y[1:]
    if op != "residual_forward":
        d, dw, db = _norm_backward(s, s["dy"].float(), h.float(), *stats)
        d = d + s["dh"].float()
        out = (*out, _dropout(s, d).to(dt), d.to(dt), dw, db)
    return out


# ---------------------------------------------------------------- the framework's calls
def _calls(s):
    import global_l2_norm_amd as G
    op, w, b, case = s["case"]["op"], s["weight"], s["bias"], s["case"]
    mask = G.DropoutMask(s["p"], s["seed"], s["step"], s["site"]) if s["p"] else None
    if op == "norm_forward":
        out = G.layer_norm_forward(s["x"], w, b, EPS, stats=case["stats"])
        return out if case["stats"] else out[:1]
    if op == "dropout_forward":
        return G.dropout_forward(s["x"], mask)
    if op == "dropout_backward":
        return G.dropout_backward(s["dy"], mask)
    grads = dict(dweight=s.get("dweight"), dbias=s.get("dbias"), accumulate=case["accumulate"])
    if op == "norm_backward":
        return G.layer_norm_backward(s["dy"], s["h"], s["mean"], s["rstd"], w, **grads)
    out = ()
    h, mean, rstd = s.get("h"), s.get("mean"), s.get("rstd")
    if op != "residual_backward":
        h, y, mean, rstd = G.residual_norm_forward(s["x"], s["residual"], w, b, EPS, mask, stats=case["stats"])
        out = (h, y, mean, rstd) if case["stats"] else (h, y)
    if op != "residual_forward":
        out = (*out, *G.residual_norm_backward(s["dy"], s["dh"], h, mean, rstd, w, mask, **grads))
    return out


def run(state):
    return _calls(state) if own else _plain(state)


def work(case):
    n, e = case["rows"] * case["size"], 4 if case["dtype"] == "f32" else 2
    w = case["size"] * (4 if case["weights"] == "f32" else 2)
    op, stats = case["op"], 8 * case["rows"] if case["stats"] else 0
    grads = w + 2 * w * (2 if case["accumulate"] else 1)  # the weight read, both gradients written, or read too
    random = 15 * n if case["p"] else 0  # ten rounds of two products and four additions or xors for eight elements
    passes = {"norm_forward": 2, "norm_backward": 3, "dropout_forward": 2, "dropout_backward": 2, "residual_forward": 4,
              "residual_backward": 5 if case["p"] else 4, "residual_step": 8 if case["p"] else 7}[op]
    rest = {"norm_forward": 2 * w + stats, "norm_backward": grads + stats, "residual_forward": 2 * w + stats,
            "residual_backward": grads + stats, "residual_step": 2 * w + grads + stats}.get(op, 0)
    sums = {"norm_forward": 8, "norm_backward": 16, "residual_forward": 9, "residual_backward": 17, "residual_step": 26}
    return {"bytes": passes * n * e + rest, "flops": sums.get(op, 1) * n + random * (2 if op == "residual_step" else 1)}


# ---------------------------------------------------------------- the definition in 64 bits
def _factors64(s, rows, size):
    """The factor 0 or s of each element, by words of an unsigned 64-bit type on the host."""
    import numpy as np
    if s["p"] == 0.0:
        return torch.ones(rows, size, dtype=torch.float64, device="cuda")
    drop = int(s["p"] * 65536 + 0.5)
    u32, m = np.uint64(32), np.uint64(0xFFFFFFFF)
    groups = -(-size // 8)
    word = [np.tile(np.arange(groups, dtype=np.uint64), rows), np.repeat(np.arange(rows, dtype=np.uint64), groups),
            np.full(rows * groups, s["site"], np.uint64), np.full(rows * groups, s["step"], np.uint64)]
    key = [s["seed"] % (1 << 32), s["seed"] // (1 << 32)]
    for i in range(10):
        keys = [np.uint64((key[0] + i * 0x9E3779B9) % (1 << 32)), np.uint64((key[1] + i * 0xBB67AE85) % (1 << 32))]
        p, q = np.uint64(0xD2511F53) * word[0], np.uint64(0xCD9E8D57) * word[2]
        word = [(q >> u32) ^ word[1] ^ keys[0], q & m, (p >> u32) ^ word[3] ^ keys[1], p & m]
    bits = np.stack([w.astype(np.uint32) for w in word], 1).astype("<u4").view("<u2")
    kept = torch.from_numpy((bits.reshape(rows, groups * 8)[:, :size] >= drop)).to("cuda")
    return kept.double() * (65536 / (65536 - drop))


def exact(case, seed):
    s, op, dt = prepare(case, seed), case["op"], DTYPES[case["dtype"]]
    v = {k: x.double() for k, x in s.items() if isinstance(x, torch.Tensor)}
    first = next(v[k] for k in ("x", "dy") if k in v)
    factor = _factors64(s, *first.shape) if not op.startswith("norm") else None
    if op.startswith("dropout"):
        return first * factor
    out = []
    h, mean, rstd = v.get("x", v.get("h")), v.get("mean"), v.get("rstd")
    if op in ("residual_forward", "residual_step"):
        out.append(v["residual"] + v["x"] * factor)
        h = out[0].to(dt).double()  # the norm is that of the stored h
    if op in ("norm_forward", "residual_forward", "residual_step"):
        mean = h.mean(1)
        rstd = ((h - mean.unsqueeze(1)).pow(2).mean(1) + EPS).rsqrt()
        out.append((h - mean.unsqueeze(1)) * rstd.unsqueeze(1) * v["weight"] + v["bias"])
        if case["stats"]:
            out += [mean, rstd]
    if op in ("norm_backward", "residual_backward", "residual_step"):
        n, g = (h - mean.unsqueeze(1)) * rstd.unsqueeze(1), v["dy"] * v["weight"]
        d = (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True)) * rstd.unsqueeze(1)
        if op != "norm_backward":
            d = d + v["dh"]
            out.append(d * factor)
        out += [d, (v["dy"] * n).sum(0) + v.get("dweight", 0.0), v["dy"].sum(0) + v.get("dbias", 0.0)]
    return tuple(out)
