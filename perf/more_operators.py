"""What is measured of the block operators: RMS norm with the residual step, with outputs and checkpoints in 8 bits; the
(gated) activation with checkpoints in 8 bits; and log probabilities of given tokens, with entropy and top alternatives.
Each forward and backward.

With ``own`` false, ``run`` computes them in elementary torch operations; with ``own`` true it makes the calls of
``global_l2_norm_amd``.  The formulas, over the rows of a matrix of `size` columns:

  norm           rstd = 1 / sqrt(sum(h^2) / size + eps), y = h rstd w
  its gradient   n = h rstd, g = dy w, dx = rstd (g - n sum(g n) / size), dw = sum over rows of dy n (added to what is
                 there when accumulating)
  residual step  h = residual + dropout(x), rounded to its type; y = norm(h).  Its gradient: dresidual = dh + the
                 norm's dx at h, dx = dropout(dresidual)
  dropout        x s where kept, else 0.  Element (r, c) takes the 16-bit half number c mod 8 (low halves first) of
                 Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) on
                 the counter (c div 8, r, site, step) under the key (seed's low word, high word), and is kept when that
                 is t = floor(65536 p + 1/2) or more; s = 65536 / (65536 - t)
  8 bits         scale = max(a / 448, 2^-112), a the largest finite magnitude of a row or of 128 of its columns;
                 q = v / scale in e4m3 (torch.float8_e4m3fn); it stands for q scale
  activation     y = act(gate) up, or act(gate); act = silu: x / (1 + exp(-x)); gelu: x (1 + erf(x / sqrt 2)) / 2;
                 gelu_tanh: x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2; relu.  dgate = dy up act'(gate),
                 dup = dy act(gate), and y again where the checkpoint stands in for it
  log probs      m = max(x), s = log(sum(exp(x - m))), log p = x - m - s, logp = log p[target], entropy = -sum(p log p);
                 dx = dlogp (1[target] - p) - dentropy p (log p + entropy), from m and s; the k largest with their
                 columns, of equal ones the lowest column first.  Rows whose target is -100 count for nothing: zeros,
                 and columns -1 with log probabilities -inf.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 128
IGNORED = -100
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
KINDS = ("silu", "gelu", "gelu_tanh", "relu")
OPS = ("norm_forward", "norm_backward", "residual_forward", "residual_backward", "residual_step",
       "activation_forward", "activation_backward", "activation_step", "pack", "unpack",
       "logp_forward", "logp_backward", "logp_step")


def _case(name, op, rows, size, dtype, weights="f32", p=0.0, stats=True, packed="", keep=False, pad=0, accumulate=False,
          kind="silu", gated=True, recompute=False, entropy=True, top=0, masked=False):
    """weights: type of weight and its gradient; stats: keep rstd, or m and s, for a backward pass; packed: y in 8 bits, a scale for
    each "row" or "block"; keep: also leave (forward), or start from (backward), a checkpoint in 8 bits; pad: columns
    between the end of a row and the next; recompute: y again in the backward pass; top: alternatives wanted; masked:
    logits of -inf (a padded vocabulary, and rows where few tokens are allowed) and rows that are not counted."""
    c = {"op": op, "rows": rows, "size": size, "dtype": dtype}
    if op.startswith(("norm", "residual")):
        c.update(weights=weights, p=p, stats=stats, packed=packed, keep=keep, pad=pad, accumulate=accumulate)
    elif op.startswith("activation"):
        c.update(kind=kind, gated=gated, keep=keep, pad=pad, recompute=recompute)
    elif op.startswith("logp"):
        c.update(entropy=entropy, stats=stats, top=top, masked=masked, pad=pad)
    else:
        c.update(packed=packed or "block", pad=pad)
    return {"name": name, **c} if name else c


def listed():
    return [
        # a block's residual add and norm for one generated token, y in 8 bits for a product of 8-bit operands
        _case("token residual 8-bit", "residual_forward", 1, 2048, "bf16", "bf16", stats=False, packed="row"),
        # the residual step of a microbatch of the 120M-parameter model in binary32, h kept in 8 bits for its gradient
        _case("120M residual kept", "residual_forward", 8192, 768, "f32", p=0.1, keep=True),
        # the same step's gradient in the 1.3B-parameter bf16 model, from h in 8 bits
        _case("1.3B residual gradient", "residual_backward", 16384, 2048, "bf16", p=0.1, keep=True),
        # a ragged batch of packed sequences, odd width, inputs that are slices of wider buffers; both directions
        _case("ragged residual step", "residual_step", 1021, 1111, "f16", p=0.25, keep=True, pad=5),
        # the gated activation of a block of that size (8/3 of 2048 columns), gate and up kept in 8 bits
        _case("1.3B gated kept", "activation_forward", 16384, 5504, "bf16", keep=True),
        # its gradient from them, with y again for the weight gradient of the product behind it
        _case("1.3B gated gradient", "activation_backward", 16384, 5504, "bf16", keep=True, recompute=True),
        # an ungated activation of odd width, both directions, kept
        _case("ragged gelu step", "activation_step", 2047, 1367, "f32", kind="gelu", gated=False, keep=True),
        # any other activation into 8 bits, for instance a product's input that its weight gradient needs ...
        _case("1.3B pack", "pack", 16384, 2048, "bf16"),
        # ... and out of them
        _case("1.3B unpack", "unpack", 16384, 2048, "bf16"),
        # eight requests' next tokens with their alternatives, a padded vocabulary, some of it not allowed
        _case("8 requests top 20", "logp_forward", 8, 131072, "bf16", stats=False, top=20, masked=True),
        # the loss of a microbatch of the 120M model: log probabilities and entropies, and their gradient
        _case("120M log probs step", "logp_step", 8192, 8449, "f32"),
        # their gradient in the 1.3B model, some tokens not counted
        _case("1.3B log probs gradient", "logp_backward", 4096, 50304, "bf16", masked=True),
    ]


def draw(rng):
    op = rng.choice(OPS)
    dtype = rng.choice(("f32", "f16", "bf16", "bf16"))
    logp = op.startswith("logp")
    top = rng.choice((1, 5, 20)) if op == "logp_forward" and rng.random() < 0.5 else 0
    size = int(round(math.exp(rng.uniform(math.log(32), math.log(131072 if logp else 16384)))))
    if rng.random() < 0.5:
        size = max(8, size // 64 * 64)
    most = (4096 * 50304 if logp else 16384 * 5504 if op.startswith("activation") else 16384 * 2048) // size
    if op.endswith("step"):
        most //= 3
    if dtype == "f32":
        most //= 2
    if top:
        most = min(most, 1 + (1 << 24) // size)
    rows = max(1, int(round(math.exp(rng.uniform(0.0, math.log(max(2, min(most, 65536))))))))
    pad = rng.choice((0, 0, 1, 8))
    dropped = rng.choice((0.05, 0.1, 0.3)) if op.startswith("residual") and rng.random() < 0.7 else 0.0
    # a step's gradient does not need y; the forward passes have it in either form
    packed = rng.choice(("row", "block")) if op in ("pack", "unpack") else rng.choice(("", "row", "block")) if op.endswith("forward") else ""
    return _case("", op, rows, size, dtype, rng.choice(("f32", dtype)), dropped, op.endswith("step") or rng.random() < 0.6, packed,
                 rng.random() < 0.6, pad, op in ("norm_backward", "residual_backward") and rng.random() < 0.5, rng.choice(KINDS),
                 rng.random() < 0.6, op != "activation_forward" and rng.random() < 0.5, rng.random() < 0.7, min(top, size),
                 rng.random() < 0.5)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, size, dt, op = case["rows"], case["size"], DTYPES[case["dtype"]], case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def matrix(scale=1.0, spread=None, shift=None, width=size):
        m = normal(rows, width + case["pad"])[:, :width].mul_(scale)
        if spread is not None:
            m.mul_(spread).add_(shift)
        return m.to(dt).contiguous() if case["pad"] == 0 else torch.empty(rows, width + case["pad"], dtype=dt, device="cuda")[:, :width].copy_(m)

    def channels(width=size):
        # channels of different spread and offset, a few of them large, as a residual stream has
        spread = 0.5 + torch.rand(width, generator=g, device="cuda")
        spread[torch.randint(0, width, (max(1, width // 256),), generator=g, device="cuda")] *= 8.0
        return spread, 0.3 * normal(width)

    s = {"case": case}
    if op.startswith(("norm", "residual")):
        wt = DTYPES[case["weights"]]
        s.update(seed=(seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 64), step=seed % 100003, site=size % 97, p=case["p"],
                 weight=(1.0 + 0.1 * normal(size)).to(wt))
        spread, shift = channels()
        if op == "norm_forward":
            s["x"] = matrix(1.0, spread, shift)
        elif op in ("residual_forward", "residual_step"):
            s["x"], s["residual"] = matrix(0.5), matrix(1.0, spread, shift)
        else:
            s["h"] = matrix(1.0, spread, shift)
            s["rstd"] = 1.0 / torch.sqrt(s["h"].float().square().sum(1) / size + EPS)
            if case["keep"]:
                s["h8"] = _pack_padded(s.pop("h").float())
        if not op.endswith("forward"):
            s["dy"] = matrix(1e-2)
            if op.startswith("residual"):
                s["dh"] = matrix(1e-2)
        if case["accumulate"]:
            s["dweight"] = normal(size).mul_(0.1).to(wt)
    elif op.startswith("activation"):
        # a product's output: gate and up are the halves of one matrix
        width = size * (2 if case["gated"] else 1)
        both = matrix(1.5, *channels(width), width)
        s["gate"], s["up"] = both[:, :size], both[:, size:] if case["gated"] else None
        if op != "activation_forward":
            s["dy"] = matrix(1e-2)
        if op == "activation_backward" and case["keep"]:
            s["gate"] = _pack_padded(s["gate"].float())
            s["up"] = _pack_padded(s["up"].float()) if case["gated"] else None
    elif op.startswith("logp"):
        # logits: most tokens unlikely, a few of each row likely
        x = matrix(2.0)
        likely = (torch.randint(0, size, (rows, 1), generator=g, device="cuda") + torch.arange(8, device="cuda") * (size // 8)) % size
        x.scatter_add_(1, likely, (4.0 + 3.0 * normal(rows, 8)).to(dt))
        allowed = size
        if case["masked"]:
            allowed = size - size // 50
            x[:, allowed:] = float("-inf")  # the padding of the vocabulary
            few = torch.rand(rows, generator=g, device="cuda") < 0.1  # rows where a grammar allows one token in 64
            x.masked_fill_(few[:, None] & (torch.arange(size, device="cuda") % 64 != 3), float("-inf"))
        s["logits"] = x
        s["targets"] = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.5, likely[:, 0] % allowed,
                                   torch.randint(0, allowed, (rows,), generator=g, device="cuda"))
        if case["masked"]:
            s["targets"] = torch.where(few, 3, s["targets"]).masked_fill(torch.rand(rows, generator=g, device="cuda") < 0.1, IGNORED)
        if op != "logp_forward":
            s["dlogp"], s["dentropy"] = -1.0 / rows + 0.1 / rows * normal(rows), 1e-2 / rows * normal(rows) if case["entropy"] else None
        if op == "logp_backward":
            _, s["entropy"], s["stats"] = _logp_rows(x, s["targets"], True)
    elif op == "pack":
        s["x"] = matrix(1.0, *channels())
    else:
        s["x8"] = _pack_padded(matrix(1.0, *channels()).float(), case["packed"])
    return s


# ---------------------------------------------------------------- the plain forms
def _pack(v, mode="block"):
    """(q, scales) of a binary32 matrix."""
    rows, size = v.shape
    group = size if mode == "row" else BLOCK
    groups = -(-size // group)
    v = torch.cat((v, v.new_zeros(rows, groups * group - size)), 1) if groups * group != size else v
    v = v.reshape(rows, groups, group)
    a = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v)).amax(2)
    scale = torch.clamp(a / 448.0, min=2.0 ** -112)
    q = (v * (1.0 / scale)[:, :, None]).to(torch.float8_e4m3fn)
    return q.reshape(rows, groups * group)[:, :size], scale


def _pack_padded(v, mode="block"):
    """As a user's program holds them: rows at a multiple of eight bytes."""
    q, scale = _pack(v, mode)
    rows, size = v.shape
    held = torch.zeros(rows, -(-size // 8) * 8, dtype=torch.uint8, device=v.device)
    held[:, :size] = q.contiguous().view(torch.uint8)
    return held.view(torch.float8_e4m3fn)[:, :size], scale


def _unpack(packed):
    q, scale = packed
    size, groups = q.shape[1], scale.shape[1]
    return q.float() * (scale if groups == 1 else scale.repeat_interleave(BLOCK, 1)[:, :size])


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
    """y (or its 8-bit form), rstd where wanted and h's checkpoint where wanted."""
    case = s["case"]
    rstd = 1.0 / torch.sqrt(h.square().sum(1) / h.shape[1] + EPS)
    y = h * rstd[:, None] * s["weight"].float()
    out = _pack(y, case["packed"]) if case["packed"] else (y.to(dt),)
    return out, rstd, _pack(h) if case["keep"] else ()


def _norm_backward(s, dy, h, rstd):
    """dx in binary32 and the weight's gradient."""
    n = h * rstd[:, None]
    g = dy * s["weight"].float()
    dx = rstd[:, None] * (g - n * ((g * n).sum(1, keepdim=True) / h.shape[1]))
    dw = (dy * n).sum(0)
    if s["case"]["accumulate"]:
        return dx, s["dweight"].copy_(s["dweight"].float() + dw)
    return dx, dw.to(s["weight"].dtype)


def _plain_norm(s):
    case, op, dt = s["case"], s["case"]["op"], DTYPES[s["case"]["dtype"]]
    out, h, rstd = (), s.get("h"), s.get("rstd")
    kept = s.get("h8")
    if not op.endswith("backward"):
        h = s["x"]
        if op.startswith("residual"):
            h = (s["residual"].float() + _dropout(s, s["x"].float())).to(dt)
            out = (h,)
        y, rstd, kept = _norm_forward(s, h.float(), dt)
        out = (*out, *y, *((rstd,) if case["stats"] else ()), *kept)
    if not op.endswith("forward"):
        d, dw = _norm_backward(s, s["dy"].float(), _unpack(kept) if case["keep"] else h.float(), rstd)
        if op.startswith("residual"):
            d = d + s["dh"].float()
            out = (*out, _dropout(s, d).to(dt))
        out = (*out, d.to(dt), dw)
    return out


def _act(kind, x):
    """act(x) and its derivative."""
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-x))
        return x * p, p * (1.0 + x * (1.0 - p))
    if kind == "gelu":
        c = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
        return x * c, c + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    if kind == "gelu_tanh":
        t = torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x))
        return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * x * x)
    return torch.clamp(x, min=0.0), (x > 0.0).float()


def _plain_activation(s):
    case, op, dt = s["case"], s["case"]["op"], DTYPES[s["case"]["dtype"]]
    out, gate, up = (), s["gate"], s["up"]
    if op != "activation_backward":
        a, b = gate.float(), up.float() if case["gated"] else None
        y = _act(case["kind"], a)[0]
        out = ((y * b if case["gated"] else y).to(dt),)
        if case["keep"]:
            gate, up = _pack(a), _pack(b) if case["gated"] else None
            out = (*out, *gate, *(up or ()))
    if op != "activation_forward":
        a = _unpack(gate) if case["keep"] else gate.float()
        y, slope = _act(case["kind"], a)
        dy = s["dy"].float()
        if case["gated"]:
            b = _unpack(up) if case["keep"] else up.float()
            out = (*out, torch.cat(((dy * b * slope).to(dt), (dy * y).to(dt)), 1))
            y = y * b
        else:
            out = (*out, (dy * slope).to(dt))
        if case["recompute"]:
            out = (*out, y.to(dt))
    return out


def _logp_rows(logits, targets, entropy):
    """log p of the targets, entropy, and m and s of each row."""
    x = logits.float()
    m = x.amax(1)
    t = x - m[:, None]
    e = torch.exp(t)
    total = e.sum(1)
    counted = targets != IGNORED
    zero = torch.zeros_like(m)
    logs = torch.log(total)
    logp = torch.where(counted, t.gather(1, targets.clamp(min=0)[:, None])[:, 0] - logs, zero)
    h = None
    if entropy:
        h = logs - torch.where(e > 0.0, t * e, torch.zeros_like(t)).sum(1) / total
        h = torch.where(counted, h, zero)
    return logp, h, torch.where(counted[:, None], torch.stack((m, logs), 1), zero[:, None])


def _plain_logp(s):
    case, op, dt = s["case"], s["case"]["op"], DTYPES[s["case"]["dtype"]]
    out, entropy, stats = (), s.get("entropy"), s.get("stats")
    counted = s["targets"] != IGNORED
    if op != "logp_backward":
        logp, entropy, stats = _logp_rows(s["logits"], s["targets"], case["entropy"])
        out = (logp, *((entropy,) if case["entropy"] else ()), *((stats,) if case["stats"] else ()))
        if case["top"]:
            value, column = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
            value, column = value[:, :case["top"]] - stats[:, :1] - stats[:, 1:], column[:, :case["top"]]
            out = (*out, torch.where(counted[:, None], value, torch.full_like(value, float("-inf"))),
                   torch.where(counted[:, None], column, torch.full_like(column, -1)))
    if op != "logp_forward":
        z = s["logits"].float() - stats[:, :1] - stats[:, 1:]
        dlogp = torch.where(counted, s["dlogp"], torch.zeros_like(s["dlogp"]))
        z = torch.where(counted[:, None], z, torch.zeros_like(z))
        p = torch.exp(z)
        d = -p * dlogp[:, None]
        if case["entropy"]:
            dh = torch.where(counted, s["dentropy"], torch.zeros_like(s["dentropy"]))
            d = d - torch.where(p > 0.0, p * (z + entropy[:, None]), torch.zeros_like(p)) * dh[:, None]
        d.scatter_add_(1, s["targets"].clamp(min=0)[:, None], dlogp[:, None])
        out = (*out, d.to(dt))
    return out


def _plain(s):
    op = s["case"]["op"]
    if op == "pack":
        return _pack(s["x"].float(), s["case"]["packed"])
    if op == "unpack":
        return _unpack(s["x8"]).to(DTYPES[s["case"]["dtype"]])
    return (_plain_activation if op.startswith("activation") else _plain_logp if op.startswith("logp") else _plain_norm)(s)


# ---------------------------------------------------------------- the framework's calls
def _parts(packed):
    return (packed.values, packed.scales) if packed is not None else ()


def _calls(s):
    import global_l2_norm_amd as G
    case, op = s["case"], s["case"]["op"]
    if op == "pack":
        return _parts(G.pack8(s["x"], case["packed"]))
    if op == "unpack":
        return G.unpack8(G.Packed8(*s["x8"]), DTYPES[case["dtype"]])
    if op.startswith("activation"):
        return _activation_calls(G, s, case, op)
    if op.startswith("logp"):
        return _logp_calls(G, s, case, op)
    w, packed = s["weight"], case["packed"] or None
    mask = G.DropoutMask(s["p"], s["seed"], s["step"], s["site"]) if s["p"] else None
    out, h, rstd = (), s.get("h"), s.get("rstd")
    kept = G.Packed8(*s["h8"]) if "h8" in s else None
    if op == "norm_forward":
        y, rstd, kept = G.rms_norm_forward(s["x"], w, EPS, packed=packed, keep=case["keep"], stats=case["stats"])
    elif op in ("residual_forward", "residual_step"):
        h, y, rstd, kept = G.residual_rms_norm_forward(s["x"], s["residual"], w, EPS, mask, packed=packed, keep=case["keep"], stats=case["stats"])
        out = (h,)
    if not op.endswith("backward"):
        out = (*out, *(_parts(y) if packed else (y,)), *((rstd,) if case["stats"] else ()), *_parts(kept))
    grads = dict(dweight=s.get("dweight"), accumulate=case["accumulate"])
    if op == "norm_backward":
        out = G.rms_norm_backward(s["dy"], kept if case["keep"] else h, rstd, w, **grads)
    elif not op.endswith("forward"):
        out = (*out, *G.residual_rms_norm_backward(s["dy"], s["dh"], kept if case["keep"] else h, rstd, w, mask, **grads))
    return out


def _activation_calls(G, s, case, op):
    out, gate, up, size = (), s["gate"], s["up"], case["size"]
    if op != "activation_backward":
        y, gate8, up8 = G.activation_forward(gate, up, case["kind"], keep=case["keep"])
        out = (y, *_parts(gate8), *_parts(up8))
        if case["keep"]:
            gate, up = gate8, up8
    elif case["keep"]:
        gate, up = G.Packed8(*gate), G.Packed8(*up) if up is not None else None
    if op == "activation_forward":
        return out
    both = to_gate = to_up = None
    if up is not None:  # the gradient of the product's output: both halves of one matrix
        both = torch.empty(case["rows"], 2 * size, dtype=s["dy"].dtype, device=s["dy"].device)
        to_gate, to_up = both[:, :size], both[:, size:]
    dgate, _, y = G.activation_backward(s["dy"], gate, up, case["kind"], recompute=case["recompute"], out_gate=to_gate, out_up=to_up)
    return (*out, dgate if both is None else both, *((y,) if case["recompute"] else ()))


def _logp_calls(G, s, case, op):
    out, entropy, stats = (), s.get("entropy"), s.get("stats")
    if op != "logp_backward":
        r = G.token_log_probs_forward(s["logits"], s["targets"], entropy=case["entropy"], top=case["top"], stats=case["stats"])
        entropy, stats = r.entropy, r.stats
        out = (r.logp, *((entropy,) if case["entropy"] else ()), *((stats,) if case["stats"] else ()),
               *((r.top_logp, r.top_ids) if case["top"] else ()))
    if op != "logp_forward":
        out = (*out, G.token_log_probs_backward(s["dlogp"], s["dentropy"], s["logits"], s["targets"], stats, entropy))
    return out


def run(state):
    return _calls(state) if own else _plain(state)


def work(case):
    rows, size, op = case["rows"], case["size"], case["op"]
    n, e = rows * size, 4 if case["dtype"] == "f32" else 2
    blocks = 4 * rows * -(-size // BLOCK)
    eight = n + blocks  # a matrix in 8 bits
    if op in ("pack", "unpack"):
        return {"bytes": n * e + n + (4 * rows if case["packed"] == "row" else blocks), "flops": 3 * n if op == "pack" else n}
    back, fore = not op.endswith("forward"), not op.endswith("backward")
    if op.startswith("logp"):
        # the logits once for each direction; a row's numbers
        return {"bytes": n * e * (fore + 2 * back) + rows * (8 + (8 + 8 * case["stats"]) * fore + 20 * back + 12 * case["top"]),
                "flops": n * ((6 if case["entropy"] else 4) * fore + (8 if case["entropy"] else 4) * back)}
    if op.startswith("activation"):
        inputs = 2 if case["gated"] else 1
        kept = inputs * eight if case["keep"] else 0
        b = f = 0
        if fore:
            b, f = b + n * e * (inputs + 1) + kept, f + 8 * n
        if back:
            b += n * e * (1 + inputs + (1 if case["recompute"] else 0)) + (kept if case["keep"] else inputs * n * e)
            f += 14 * n
        return {"bytes": b, "flops": f}
    residual = op.startswith("residual")
    w = size * (4 if case["weights"] == "f32" else 2)
    drop = 1 if case["p"] else 0
    b, f = w, 0
    if fore:
        b += n * e * (3 if residual else 1) + (n * e if not case["packed"] else n + 4 * rows if case["packed"] == "row" else eight)
        b += (4 * rows if case["stats"] else 0) + (eight if case["keep"] else 0)
        f += (5 + 15 * drop) * n
    if back:
        b += (eight if case["keep"] else n * e) + n * e * (2 + (1 + drop if residual else 0)) + 4 * rows
        b += w * (2 if case["accumulate"] else 1)
        f += (9 + 15 * drop) * n
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_eight(v, mode):
    """v / scale, what an 8-bit value is before its rounding, and the scales."""
    rows, size = v.shape
    if mode == "row":
        scale = v.abs().max(1, keepdim=True).values.div(448.0).clamp_min(2.0 ** -112)
        return [v / scale, scale]
    q, scales = torch.empty_like(v), []
    for first in range(0, size, BLOCK):
        part = v[:, first:first + BLOCK]
        scales.append(part.abs().max(1).values.div(448.0).clamp_min(2.0 ** -112))
        q[:, first:first + BLOCK] = part / scales[-1].unsqueeze(1)
    return [q, torch.stack(scales, 1)]


def _exact_value(held):
    q, scale = held[0].double(), held[1].double()
    if scale.shape[1] == 1:
        return q * scale
    column = torch.arange(q.shape[1], device=q.device) // BLOCK
    return q * scale[:, column]


def _factors64(s, rows, size):
    """The factor 0 or s of each element, by words of an unsigned 64-bit type on the host."""
    import numpy as np
    if s["p"] == 0.0:
        return 1.0
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


def _exact_norm(s, case, op, dt):
    w, out = s["weight"].double(), []
    factor = _factors64(s, case["rows"], case["size"]) if op.startswith("residual") else 1.0
    rstd = s["rstd"].double() if "rstd" in s else None
    h = _exact_value(s["h8"]) if "h8" in s else s["h"].double() if "h" in s else None
    if not op.endswith("backward"):
        h = s["x"].double()
        if op.startswith("residual"):
            out.append(s["residual"].double() + h * factor)
            # the norm is that of the stored h: the sum in binary32, as the stored h is rounded from it
            h = (s["residual"].float() + (s["x"].float() * torch.as_tensor(factor, device="cuda").float())).to(dt).double()
        rstd = (h.pow(2).mean(1) + EPS).rsqrt()
        y = h * rstd.unsqueeze(1) * w
        out += _exact_eight(y, case["packed"]) if case["packed"] else [y]
        if case["stats"]:
            out.append(rstd)
        if case["keep"]:
            held = _exact_eight(h, "block")
            out += held
            # what the gradient starts from: the rounded values
            h = _exact_value(_pack(h.float()))
    if not op.endswith("forward"):
        dy = s["dy"].double()
        n, g = h * rstd.unsqueeze(1), dy * w
        d = (g - n * (g * n).mean(1, keepdim=True)) * rstd.unsqueeze(1)
        if op.startswith("residual"):
            d = d + s["dh"].double()
            out.append(d * factor)
        out += [d, (dy * n).sum(0) + (s["dweight"].double() if case["accumulate"] else 0.0)]
    return tuple(out)


def _exact_act(kind, x):
    if kind == "relu":
        return x.relu(), x.gt(0).double()
    if kind == "silu":
        p = torch.sigmoid(x)
        return x * p, p + x * p * torch.sigmoid(-x)
    if kind == "gelu":
        c = torch.special.ndtr(x)
        return x * c, c + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    u = k * (x + 0.044715 * x ** 3)
    c = torch.sigmoid(2 * u)  # (1 + tanh(u)) / 2
    return x * c, c + x * 2 * c * torch.sigmoid(-2 * u) * k * (1 + 3 * 0.044715 * x ** 2)


def _exact_activation(s, case, op):
    out = []
    gate, up = s["gate"], s["up"]
    if op == "activation_backward" and case["keep"]:
        a, b = _exact_value(gate), _exact_value(up) if up is not None else None
    else:
        a, b = gate.double(), up.double() if up is not None else None
    if op != "activation_backward":
        y = _exact_act(case["kind"], a)[0]
        out.append(y if b is None else y * b)
        if case["keep"]:
            out += _exact_eight(a, "block")
            a = _exact_value(_pack(a.float()))
            if b is not None:
                out += _exact_eight(b, "block")
                b = _exact_value(_pack(b.float()))
    if op != "activation_forward":
        y, slope = _exact_act(case["kind"], a)
        dy = s["dy"].double()
        out.append(dy * slope if b is None else torch.cat((dy * b * slope, dy * y), 1))
        if case["recompute"]:
            out.append(y if b is None else y * b)
    return tuple(out)


def _exact_logp(s, case, op):
    x = s["logits"].double()
    target, counted = s["targets"].clamp_min(0).unsqueeze(1), s["targets"].ne(IGNORED)
    z = torch.log_softmax(x, 1)
    p = z.exp()
    h = -torch.where(p.gt(0), p * z, 0.0).sum(1) * counted
    out = []
    if op != "logp_backward":
        out.append(z.gather(1, target).squeeze(1).masked_fill(~counted, 0.0))
        if case["entropy"]:
            out.append(h)
        if case["stats"]:
            m = x.max(1).values
            out.append(torch.stack((m, x.logsumexp(1) - m), 1).masked_fill(~counted.unsqueeze(1), 0.0))
        if case["top"]:
            out += [z.sort(1, descending=True).values[:, :case["top"]].masked_fill(~counted.unsqueeze(1), -math.inf), None]
    if op != "logp_forward":
        if op == "logp_backward":
            z = x - s["stats"].double().sum(1, keepdim=True)
            p, h = z.exp(), s["entropy"].double()
        onto = torch.zeros_like(p).scatter_(1, target, 1.0)
        d = (onto - p) * s["dlogp"].double().unsqueeze(1)
        if case["entropy"]:
            d -= torch.where(p.gt(0), p * (z + h.unsqueeze(1)), 0.0) * s["dentropy"].double().unsqueeze(1)
        out.append(torch.where(counted.unsqueeze(1), d, 0.0))
    return tuple(out)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "pack":
        return tuple(_exact_eight(s["x"].double(), case["packed"]))
    if op == "unpack":
        return _exact_value(s["x8"])
    if op.startswith("activation"):
        return _exact_activation(s, case, op)
    if op.startswith("logp"):
        return _exact_logp(s, case, op)
    return _exact_norm(s, case, op, DTYPES[case["dtype"]])
