"""Cases and plain forms of root-mean-square norm with the residual's addition
(16- and 32-bit rows, and rows of 8-bit codes with block scales) and of the
gated feed-forward block that reads its rows.

Over rows t, hidden columns k and features f:

    s = x + residual,  q = (mean_k s^2 + eps)^(-1/2),  y = s q w
    G = X Wg^T,  U = X Wu^T,  A = act(G) U

``rms_norm``            x, residual -> y, s, q
``rms_norm_backward``   dy, s, q, ds -> dx = ds + q (g - h mean_k(g h)), dw = sum_t dy h
                        for h = s q and g = dy w
``rms_norm_mx``         x, residual -> codes, scales, s: y in blocks of 32 columns,
                        scale = 2^e with the least e for which max|y| <= 448 2^e,
                        codes = E4M3(y / scale)
``gated_forward``       x, Wg, Wu -> A (for training also G and U)
``gated_backward``      dA, x, G, U, Wg, Wu -> dX, dWg, dWu
                        through dG = dA U act'(G) and dU = dA act(G)
``gated_forward_mx``    codes and scales of x, Wg and Wu -> A
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
NORMS = ("rms", "rms_mx", "rms_backward")
GATED = ("gated", "gated_mx", "gated_backward")
ACTIVATIONS = ("silu", "gelu", "gelu_tanh")


def _rms(name, op, rows, hidden, dtype="bf16", param="fp32", pitch=0, residual=True):
    """residual: whether the residual stream is added (backward: whether its
    gradient arrives too).  pitch: elements between rows beyond hidden."""
    c = {"op": op, "rows": rows, "hidden": hidden, "dtype": dtype, "param": param, "pitch": pitch,
         "residual": residual}
    return dict(c, name=name) if name else c


def _gated(name, op, rows, hidden, features, dtype="bf16", activation="silu", pitch=0,
           save=False):
    """save: the forward pass also returns both projections, as training keeps them."""
    c = {"op": op, "rows": rows, "hidden": hidden, "features": features, "dtype": dtype,
         "activation": activation, "pitch": pitch}
    if op == "gated":
        c["save"] = save
    return dict(c, name=name) if name else c


def listed():
    return [
        # One token of a generated sequence: launch latency.
        _rms("rms_1x2560", "rms", 1, 2560, "bf16", "bf16"),
        # A training micro-batch.
        _rms("rms_16384x3584", "rms", 16384, 3584),
        # A ragged batch of prompts, served in 8 bits.
        _rms("rms_mx_1001x1120_f16", "rms_mx", 1001, 1120, "fp16", "fp16"),
        # A full batch of prompts.
        _rms("rms_mx_8192x2560", "rms_mx", 8192, 2560, "bf16", "bf16"),
        # A short odd batch out of a wider buffer, full precision.
        _rms("rms_back_777x2567_f32", "rms_backward", 777, 2567, "fp32", "fp32", pitch=9,
             residual=False),
        # The largest hidden state, with the residual stream's gradient.
        _rms("rms_back_32768x12288", "rms_backward", 32768, 12288),
        # One token of a generated sequence: both weights are read for it.
        _gated("gated_1_2560x10240", "gated", 1, 2560, 10240),
        # The forward pass of a training step.
        _gated("gated_8192_2560x10240", "gated", 8192, 2560, 10240, save=True),
        # A small odd layer.
        _gated("gated_back_999_1111x1030_f16", "gated_backward", 999, 1111, 1030, "fp16", "gelu"),
        # The backward pass of that training step.
        _gated("gated_back_8192_2560x10240", "gated_backward", 8192, 2560, 10240),
        # Four sequences, a token each, weights in 8 bits.
        _gated("gated_mx_4_3584x14336", "gated_mx", 4, 3584, 14336),
        # Long prompts, weights in 8 bits.
        _gated("gated_mx_16384_3584x14336", "gated_mx", 16384, 3584, 14336),
    ]


def _size(rng, low, high, step=0):
    """A size spread over its logarithm: one in three odd, the others whole
    multiples of 8 (or 64) where there is room; all multiples of `step` if given."""
    n = max(low, min(high, round(low * (high / low) ** rng.random())))
    if step:
        return max(step, n // step * step)
    kind = rng.randrange(3)
    unit = 64 if kind == 0 else 8
    if kind < 2 and n >= 2 * unit:
        return n // unit * unit
    return n if n % 2 or n == high else n + 1


def draw(rng):
    if rng.random() < 0.5:
        op = NORMS[rng.randrange(3)]
        dtype = ("bf16", "bf16", "fp16", "fp32")[rng.randrange(4)]
        hidden = _size(rng, 32, 12288, BLOCK if op == "rms_mx" else 0)
        return _rms(None, op, _size(rng, 1, 32768 if hidden <= 8192 else 16384), hidden, dtype,
                    (dtype, "fp32")[rng.randrange(2)], (0, 0, 8, 5)[rng.randrange(4)],
                    rng.random() < 0.7)
    op = GATED[rng.randrange(3)]
    step = BLOCK if op == "gated_mx" else 0
    hidden, features = _size(rng, 32, 8192, step), _size(rng, 32, 16384)
    most = (8192 * 2560 * 10240 if op != "gated_mx" else 16384 * 3584 * 14336)
    rows = _size(rng, 1, min(32768, max(2, most // (hidden * features))))
    return _gated(None, op, rows, hidden, features, ("bf16", "bf16", "fp16")[rng.randrange(3)],
                  ACTIVATIONS[rng.randrange(3)],
                  0 if op == "gated_mx" else (0, 0, 8, 5)[rng.randrange(4)],
                  op == "gated" and rng.random() < 0.5)


# --------------------------------------------------------------- inputs --

def _rows(rows, width, pitch, dtype, scale, gen):
    """[rows, width] of N(0, scale), rows width + pitch apart."""
    full = torch.empty(rows, width + pitch, dtype=torch.float32, device="cuda")
    full.normal_(0.0, scale, generator=gen)
    return full.to(dtype)[:, :width]


def _stream(case, gen):
    """A residual stream: rows of different size, a few outlier channels."""
    rows, hidden = case["rows"], case["hidden"]
    full = torch.empty(rows, hidden + case["pitch"], device="cuda").normal_(generator=gen)
    full.mul_(torch.empty(rows, 1, device="cuda").uniform_(0.5, 2.0, generator=gen))
    full[:, torch.randint(0, hidden, (4,), generator=gen, device="cuda")] *= 20.0
    return full.to(TYPES[case["dtype"]])[:, :hidden]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rows, hidden, op, dtype = case["rows"], case["hidden"], case["op"], TYPES[case["dtype"]]
    s = {"case": case}
    if op in NORMS:
        s["weight"] = torch.empty(hidden, device="cuda").normal_(1.0, 0.1, generator=gen).to(
            TYPES[case["param"]])
        s["x"] = _stream(case, gen)
        s["residual"] = None
        if op == "rms_backward":
            s["dy"] = _rows(rows, hidden, case["pitch"], dtype, 1e-2, gen)
            s["rstd"] = _rstd(s["x"].float()).flatten()
            if case["residual"]:
                s["residual"] = _rows(rows, hidden, 0, dtype, 1e-2, gen)
        elif case["residual"]:
            # What the layer adds to the stream.
            s["residual"] = _rows(rows, hidden, 0, dtype, 0.5, gen)
        return s
    features = case["features"]
    x = _rows(rows, hidden, case["pitch"], dtype, 1.0, gen)
    weights = [_rows(features, hidden, 0, dtype, hidden ** -0.5, gen) for _ in range(2)]
    if op == "gated_mx":
        s["x"], s["gate_weight"], s["up_weight"] = (_mx(t.float()) for t in (x, *weights))
        return s
    s.update(x=x, gate_weight=weights[0], up_weight=weights[1])
    if op == "gated_backward":
        s["gate"], s["up"] = (_rows(rows, features, 0, dtype, 1.0, gen) for _ in range(2))
        s["da"] = _rows(rows, features, case["pitch"], dtype, 1e-2, gen)
    return s


# ----------------------------------------------------------- plain forms --

def _rstd(x):
    return 1.0 / (x * x).mean(1, keepdim=True).add(EPS).sqrt()


def _mx(y):
    """(codes, scales), bytes, of a float32 [rows, width]."""
    blocks = y.reshape(y.shape[0], -1, BLOCK)
    part, exponent = torch.frexp(blocks.abs().amax(2))
    # max = part 2^exponent, 448 = 0.875 2^9
    e = torch.where(part > 0.875, exponent - 8, exponent - 9)
    e = torch.where(part == 0, -127, e).clamp_(min=-127).to(torch.int32)
    codes = torch.ldexp(blocks, -e[:, :, None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).reshape(y.shape), (e + 127).to(torch.uint8)


def _mx_values(pair):
    codes, scales = pair
    scale = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.to(torch.int32) - 127)
    values = codes.view(torch.float8_e4m3fn).float().view(*scales.shape, BLOCK)
    return (values * scale[:, :, None]).view(codes.shape)


def _as_values(codes, scales):
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _activation(g, kind):
    """act(g) and its derivative."""
    if kind == "silu":
        p = 1.0 / (1.0 + (-g).exp())
        return g * p, p * (1.0 + g * (1.0 - p))
    if kind == "gelu":
        p = 0.5 * (1.0 + (g * 0.5 ** 0.5).erf())
        return g * p, p + g * (-0.5 * g * g).exp() * (2.0 * math.pi) ** -0.5
    c = (2.0 / math.pi) ** 0.5
    th = (c * (g + 0.044715 * g * g * g)).tanh()
    slope = c * (1.0 + 3 * 0.044715 * g * g)
    return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * slope


def _plain_norm(s):
    op, x, w = s["case"]["op"], s["x"].float(), s["weight"].float()
    if op == "rms_backward":
        dy, q = s["dy"].float(), s["rstd"][:, None]
        h, g = x * q, dy * w
        dx = q * (g - h * (g * h).mean(1, keepdim=True))
        if s["residual"] is not None:
            dx = dx + s["residual"].float()
        return dx.to(s["x"].dtype), (dy * h).sum(0).to(s["weight"].dtype)
    total = []
    if s["residual"] is not None:
        x = x + s["residual"].float()
        total = [x.to(s["x"].dtype)]
    q = _rstd(x)
    y = x * q * w
    if op == "rms_mx":
        return [*_as_values(*_mx(y)), *total]
    return [y.to(s["x"].dtype), *total, q.flatten()]


def _plain_gated(s):
    case = s["case"]
    dtype, kind = TYPES[case["dtype"]], case["activation"]
    if case["op"] == "gated_backward":
        x, wg, wu = s["x"].float(), s["gate_weight"].float(), s["up_weight"].float()
        da = s["da"].float()
        act, slope = _activation(s["gate"].float(), kind)
        dg, du = da * s["up"].float() * slope, da * act
        dx = dg @ wg + du @ wu
        return dx.to(dtype), (dg.t() @ x).to(dtype), (du.t() @ x).to(dtype)
    value = _mx_values if case["op"] == "gated_mx" else torch.Tensor.float
    x = value(s["x"])
    gate, up = x @ value(s["gate_weight"]).t(), x @ value(s["up_weight"]).t()
    out = (_activation(gate, kind)[0] * up).to(dtype)
    return (out, gate.to(dtype), up.to(dtype)) if case.get("save") else out


def _own(s):
    case = s["case"]
    op = case["op"]
    if op in NORMS:
        from gradients_taco_compress_amd import norm
        if op == "rms_backward":
            return norm.rms_norm_backward(s["dy"], s["x"], s["rstd"], s["weight"],
                                          dtotal=s["residual"])
        if op == "rms_mx":
            codes, scales, total = norm.rms_norm_mx(s["x"], s["weight"], EPS,
                                                    residual=s["residual"])
            return [*_as_values(codes, scales), *([] if total is None else [total])]
        y, total, rstd = norm.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
        return [y, rstd] if total is None else [y, total, rstd]
    from gradients_taco_compress_amd import gated
    kind = case["activation"]
    if op == "gated_mx":
        return gated.gated_forward_mx(s["x"], s["gate_weight"], s["up_weight"], kind,
                                      dtype=TYPES[case["dtype"]])
    if op == "gated_backward":
        return gated.gated_backward(s["da"], s["x"], s["gate"], s["up"], s["gate_weight"],
                                    s["up_weight"], kind)
    return gated.gated_forward(s["x"], s["gate_weight"], s["up_weight"], kind, save=case["save"])


def run(state):
    if own:
        return _own(state)
    return _plain_norm(state) if state["case"]["op"] in NORMS else _plain_gated(state)


def work(case):
    """Each input read once, each output written once."""
    rows, hidden, op = case["rows"], case["hidden"], case["op"]
    e, n = SIZE[case["dtype"]], case["rows"] * case["hidden"]
    if op in NORMS:
        p, more = SIZE[case["param"]], 1 if case["residual"] else 0
        if op == "rms":
            return {"bytes": (2 + 2 * more) * n * e + hidden * p + 4 * rows, "flops": (4 + more) * n}
        if op == "rms_mx":
            return {"bytes": (1 + 2 * more) * n * e + n + n // BLOCK + hidden * p,
                    "flops": (6 + more) * n}
        return {"bytes": (3 + more) * n * e + 2 * hidden * p + 4 * rows, "flops": (9 + more) * n}
    features = case["features"]
    a = rows * features
    if op == "gated_mx":
        codes = n + 2 * features * hidden
        return {"bytes": codes + codes // BLOCK + a * e, "flops": 4 * n * features + 6 * a}
    if op == "gated":
        return {"bytes": (n + 2 * features * hidden + a * (3 if case["save"] else 1)) * e,
                "flops": 4 * n * features + 6 * a}
    return {"bytes": (2 * n + 4 * features * hidden + 3 * a) * e,
            "flops": 8 * n * features + 12 * a}


# ------------------------------------------------- the definition, 64 bits --

def _e4m3_64(v):
    """The E4M3 value nearest to each float64 (ties to the even code)."""
    exponent = torch.frexp(v)[1].sub(1).clamp_(min=-6)
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return (torch.round(v / step) * step).clamp_(-448.0, 448.0)


def _exact_norm(s):
    op, x, w = s["case"]["op"], s["x"].double(), s["weight"].double()
    hidden = x.shape[1]
    if op == "rms_backward":
        # The pass is given the statistics in 32 bits.
        q, dy = s["rstd"].double(), s["dy"].double()
        h = x.mul_(q[:, None])
        dw = torch.linalg.vecdot(dy, h, dim=0)
        # Rows of the norm's Jacobian: q (I - h h^T / K).
        g = dy.mul_(w)
        g.sub_((torch.linalg.vecdot(g, h, dim=1) / hidden)[:, None] * h).mul_(q[:, None])
        return g if s["residual"] is None else g.add_(s["residual"].double()), dw
    total = []
    if s["residual"] is not None:
        x = x + s["residual"].double()
        total = [x]
    q = torch.rsqrt(torch.linalg.vector_norm(x, dim=1) ** 2 / hidden + EPS)
    y = x * w * q[:, None]
    if op == "rms":
        return [y, *total, q]
    blocks = y.view(y.shape[0], hidden // BLOCK, BLOCK)
    e = torch.ceil(torch.log2(torch.linalg.vector_norm(blocks, ord=math.inf, dim=2) / 448.0))
    scale = torch.exp2(e.clamp_(min=-127.0))
    return [_e4m3_64(blocks / scale[:, :, None]).view(y.shape), scale, *total]


def _phi(g, kind):
    """act(g) / g and act'(g)."""
    if kind == "silu":
        p = torch.sigmoid(g)
        return p, torch.addcmul(p, g * p, torch.sigmoid(-g))
    if kind == "gelu":
        p = torch.special.ndtr(g)
        return p, torch.addcmul(p, g, torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi))
    # (1 + tanh(z)) / 2 = sigmoid(2 z)
    c = math.sqrt(8 / math.pi)
    p = torch.sigmoid(c * (g + 0.044715 * g ** 3))
    return p, p + g * p * (1 - p) * c * (1 + 0.134145 * g.square())


def _double(pair):
    codes, scales = pair
    exponent = scales.double().sub_(127.0).repeat_interleave(BLOCK, 1)
    return codes.view(torch.float8_e4m3fn).double().mul_(torch.exp2(exponent))


def _exact_gated(s):
    case = s["case"]
    kind = case["activation"]
    value = _double if case["op"] == "gated_mx" else torch.Tensor.double
    x, wg, wu = value(s["x"]), value(s["gate_weight"]), value(s["up_weight"])
    if case["op"] == "gated_backward":
        gate, da = s["gate"].double(), s["da"].double()
        p, slope = _phi(gate, kind)
        both = torch.cat([slope.mul_(da).mul_(s["up"].double()), gate.mul_(p).mul_(da)], 1)
        dx = torch.mm(both, torch.cat([wg, wu], 0))
        return (dx, *torch.mm(both.t(), x).chunk(2, 0))
    gate, up = torch.mm(x, wg.t()), torch.mm(x, wu.t())
    out = _phi(gate, kind)[0] * gate * up
    return (out, gate, up) if case.get("save") else out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] in NORMS else _exact_gated(s)
