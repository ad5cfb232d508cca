"""Cases and plain forms of the layer-norm operators and of the 8-bit activation
checkpoint that serves both the norm's backward pass and the weight gradient
of the linear layer behind it.

Over rows t and hidden columns k, with weight w, bias b and eps:

    m = mean_k x,  r = (mean_k (x - m)^2 + eps)^(-1/2),  h = (x - m) r,  y = h w + b

``layer_norm``                      x -> y, m, r
``layer_norm_backward``             dy, x, m, r -> dx, dw, db
``layer_norm_checkpoint``           x -> y, codes, r      codes = E4M3(S h)
``layer_norm_checkpoint_backward``  dy, codes, r -> dx, dw, db
``checkpoint_weight_grad``          dy, codes -> dW = dy^T y, db = sum_t dy

with dx = r (g - mean_k g - h mean_k (g h)) for g = dy w, dw = sum_t dy h and
db = sum_t dy; in the last two h = decode(codes) / S and y = h w + b.
S = 2^p, p the largest integer with hidden * 4^p <= 448^2: as sum_k h^2 <=
hidden, S h never leaves E4M3's range.
"""
import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
OPS = ("norm", "norm_backward", "checkpoint", "checkpoint_backward", "weight_grad")


def _case(name, op, rows, hidden, dtype="bf16", param="fp32", pitch=0, out_features=0,
          grad="same", accumulate=False):
    """pitch: elements between rows of the activations beyond hidden (a slice
    of a wider tensor).  grad: type of dW (that of dy, or fp32)."""
    c = {"op": op, "rows": rows, "hidden": hidden, "dtype": dtype, "param": param, "pitch": pitch}
    if op == "weight_grad":
        c.update(out_features=out_features, grad=grad, accumulate=accumulate)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One token of a generated sequence: launch latency.
        _case("norm_1x2560", "norm", 1, 2560, "bf16", "bf16"),
        # A training micro-batch, 4 sequences of 2048 tokens.
        _case("norm_8192x2560", "norm", 8192, 2560),
        # A small full-precision model's backward pass.
        _case("norm_back_2048x1024_f32", "norm_backward", 2048, 1024, "fp32", "fp32"),
        # Full-width backward pass.
        _case("norm_back_16384x3584", "norm_backward", 16384, 3584),
        # The checkpointing forward pass of the same micro-batch.
        _case("ckpt_16384x3584", "checkpoint", 16384, 3584),
        # A packed batch of odd length, odd width, fp16.
        _case("ckpt_1001x1111_f16", "checkpoint", 1001, 1111, "fp16", "fp16"),
        # A short odd batch out of a wider buffer.
        _case("ckpt_back_777x2568", "checkpoint_backward", 777, 2568, "bf16", "bf16", pitch=24),
        # The largest hidden state.
        _case("ckpt_back_32768x12288", "checkpoint_backward", 32768, 12288),
        # A short, small layer: few output tiles and a long sum.
        _case("wgrad_2048_1024x1024", "weight_grad", 2048, 1024, out_features=1024),
        # The first MLP matrix of the micro-batch above.
        _case("wgrad_8192_10240x2560", "weight_grad", 8192, 2560, out_features=10240),
        # Odd everything, with a gradient in full precision.
        _case("wgrad_999_1030x1111_f16", "weight_grad", 999, 1111, "fp16", "fp16",
              out_features=1030, grad="fp32"),
        # One tensor-parallel shard of the widest layer, added into the
        # float32 gradient that micro-batches share.
        _case("wgrad_32768_1536x12288_acc", "weight_grad", 32768, 12288, out_features=1536,
              grad="fp32", accumulate=True),
    ]


def _size(rng, low, high):
    """A size spread over its logarithm: one in three odd, the others whole
    multiples of 8 (or 64) where there is room."""
    n = max(low, min(high, round(low * (high / low) ** rng.random())))
    kind = rng.randrange(3)
    step = 64 if kind == 0 else 8
    if kind < 2 and n >= 2 * step:
        return n // step * step
    return n if n % 2 or n == high else n + 1


def draw(rng):
    op = OPS[rng.randrange(len(OPS))]
    if op == "weight_grad":
        dtype = ("bf16", "bf16", "fp16")[rng.randrange(3)]
        grad = ("same", "fp32")[rng.randrange(2)]
        out = _size(rng, 32, 12288)
        hidden = _size(rng, 32, 12288)
        top = min(32768, max(2, (32768 * 1536 * 12288) // (out * hidden)))
        return _case(None, op, _size(rng, 1, top), hidden, dtype, (dtype, "fp32")[rng.randrange(2)],
                     (0, 0, 8, 5)[rng.randrange(4)], out, grad,
                     grad == "fp32" and rng.random() < 0.5)
    dtype = ("bf16", "bf16", "fp16", "fp32")[rng.randrange(4)]
    hidden = _size(rng, 8, 12288)
    return _case(None, op, _size(rng, 1, 32768 if hidden <= 8192 else 16384), hidden, dtype,
                 (dtype, "fp32")[rng.randrange(2)], (0, 0, 8, 5)[rng.randrange(4)])


def _scale(hidden):
    p = 16
    while (hidden << (2 * p + 32)) > (448 * 448 << 32):
        p -= 1
    return 2.0 ** p


def _rows(rows, width, pitch, dtype, scale, gen):
    """[rows, width] of N(0, scale), rows width + pitch apart."""
    full = torch.empty(rows, width + pitch, dtype=torch.float32, device="cuda")
    full.normal_(0.0, scale, generator=gen)
    return full.to(dtype)[:, :width]


def _activation(case, gen):
    """A residual stream: rows of different size and mean, a few outlier channels."""
    rows, hidden = case["rows"], case["hidden"]
    x = _rows(rows, hidden, case["pitch"], torch.float32, 1.0, gen)
    level = torch.empty(rows, 1, device="cuda").uniform_(0.5, 2.0, generator=gen)
    mean = torch.empty(rows, 1, device="cuda").normal_(0.0, 0.2, generator=gen)
    x.mul_(level).add_(mean)
    outlier = torch.randint(0, hidden, (4,), generator=gen, device="cuda")
    x[:, outlier] *= 20.0
    return _keep_pitch(x, TYPES[case["dtype"]])


def _keep_pitch(x, dtype):
    full = torch.as_strided(x, (x.shape[0], x.stride(0)), (x.stride(0), 1))
    return full.to(dtype)[:, :x.shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rows, hidden = case["rows"], case["hidden"]
    dtype, param = TYPES[case["dtype"]], TYPES[case["param"]]
    s = {"case": case,
         "weight": torch.empty(hidden, device="cuda").normal_(1.0, 0.1, generator=gen).to(param),
         "bias": torch.empty(hidden, device="cuda").normal_(0.0, 0.1, generator=gen).to(param)}
    op = case["op"]
    x = _activation(case, gen)
    if op in ("norm", "checkpoint"):
        s["x"] = x
        return s
    width = case["out_features"] if op == "weight_grad" else hidden
    s["dy"] = _rows(rows, width, case["pitch"], dtype, 1e-2, gen)
    h, mean, rstd = _normalise(x.float())
    if op == "norm_backward":
        s.update(x=x, mean=mean.flatten(), rstd=rstd.flatten())
        return s
    s.update(codes=(h * _scale(hidden)).to(torch.float8_e4m3fn).view(torch.uint8),
             rstd=rstd.flatten())
    if op == "weight_grad":
        s["out_dtype"] = torch.float32 if case["grad"] == "fp32" else dtype
        if case["accumulate"]:
            s["acc"] = _rows(width, hidden, 0, torch.float32, 1e-2 * rows ** 0.5, gen)
    return s


# ----------------------------------------------------------- plain forms --

def _normalise(x):
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1.0 / (d * d).mean(1, keepdim=True).add(EPS).sqrt()
    return d * rstd, mean, rstd


def _decoded(s):
    return s["codes"].view(torch.float8_e4m3fn).float() / _scale(s["case"]["hidden"])


def _norm_gradients(s, h, rstd):
    dy, w = s["dy"].float(), s["weight"].float()
    g = dy * w
    c1 = g.mean(1, keepdim=True)
    c2 = (g * h).mean(1, keepdim=True)
    dx = rstd * (g - c1 - h * c2)
    kind = s["weight"].dtype
    return dx.to(s["dy"].dtype), (dy * h).sum(0).to(kind), dy.sum(0).to(kind)


def _plain(s):
    op = s["case"]["op"]
    if op in ("norm", "checkpoint"):
        h, mean, rstd = _normalise(s["x"].float())
        y = (h * s["weight"].float() + s["bias"].float()).to(s["x"].dtype)
        if op == "norm":
            return y, mean.flatten(), rstd.flatten()
        return y, (h * _scale(s["case"]["hidden"])).to(torch.float8_e4m3fn), rstd.flatten()
    if op == "norm_backward":
        rstd = s["rstd"][:, None]
        return _norm_gradients(s, (s["x"].float() - s["mean"][:, None]) * rstd, rstd)
    if op == "checkpoint_backward":
        return _norm_gradients(s, _decoded(s), s["rstd"][:, None])
    y = _decoded(s) * s["weight"].float() + s["bias"].float()
    dy = s["dy"].float()
    grad = dy.t().contiguous() @ y
    db = dy.sum(0)
    if s["case"]["accumulate"]:
        s["acc"] += grad
        return s["acc"], db
    return grad.to(s["out_dtype"]), db


def _own(s):
    from gradients_taco_compress_amd import norm
    op = s["case"]["op"]
    if op == "norm":
        return norm.layer_norm(s["x"], s["weight"], s["bias"], EPS)
    if op == "checkpoint":
        y, codes, rstd = norm.layer_norm_checkpoint(s["x"], s["weight"], s["bias"], EPS)
        return y, codes.view(torch.float8_e4m3fn), rstd
    if op == "norm_backward":
        return norm.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
    if op == "checkpoint_backward":
        return norm.layer_norm_checkpoint_backward(s["dy"], s["codes"], s["rstd"], s["weight"])
    if s["case"]["accumulate"]:
        return norm.checkpoint_weight_grad(s["dy"], s["codes"], s["weight"], s["bias"],
                                           out=s["acc"], accumulate=True)
    return norm.checkpoint_weight_grad(s["dy"], s["codes"], s["weight"], s["bias"],
                                       dtype=s["out_dtype"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    """Each input read once, each output written once."""
    rows, hidden, op = case["rows"], case["hidden"], case["op"]
    e, p, n = SIZE[case["dtype"]], SIZE[case["param"]], case["rows"] * case["hidden"]
    if op == "norm":
        return {"bytes": 2 * n * e + 2 * hidden * p + 8 * rows, "flops": 8 * n}
    if op == "checkpoint":
        return {"bytes": 2 * n * e + n + 2 * hidden * p + 4 * rows, "flops": 9 * n}
    if op == "norm_backward":
        return {"bytes": 3 * n * e + 3 * hidden * p + 8 * rows, "flops": 14 * n}
    if op == "checkpoint_backward":
        return {"bytes": 2 * n * e + n + 3 * hidden * p + 4 * rows, "flops": 13 * n}
    out = case["out_features"]
    g = 4 if case["grad"] == "fp32" else e
    return {"bytes": rows * out * e + n + out * hidden * g * (2 if case["accumulate"] else 1)
            + 4 * out + 2 * hidden * p, "flops": 2 * n * out + rows * out}


# ------------------------------------------------- the definition, 64 bits --

def _e4m3_64(v):
    """The E4M3 value nearest to each float64 (ties to the even code)."""
    exponent = torch.frexp(v)[1].sub(1).clamp_(min=-6)
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return (torch.round(v / step) * step).clamp_(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    op, hidden = case["op"], case["hidden"]
    w, b = s["weight"].double(), s["bias"].double()
    if op in ("norm", "checkpoint", "norm_backward"):
        x = s["x"].double()
        total = x.sum(1)
        mean = total / hidden
        if op == "norm_backward":
            # The pass is given the statistics in 32 bits.
            mean, rstd = s["mean"].double(), s["rstd"].double()
        else:
            x2 = torch.linalg.vector_norm(x - mean[:, None], dim=1) ** 2
            rstd = torch.rsqrt(x2 / hidden + EPS)
        x.sub_(mean[:, None]).mul_(rstd[:, None])
        if op == "norm":
            return torch.addcmul(b, x, w), mean, rstd
        if op == "checkpoint":
            return torch.addcmul(b, x, w), _e4m3_64(x * _scale(hidden)), rstd
        h = x
    else:
        h = s["codes"].view(torch.float8_e4m3fn).double() * (1.0 / _scale(hidden))
    dy = s["dy"].double()
    db = torch.ones(case["rows"], dtype=torch.float64, device="cuda") @ dy
    if op == "weight_grad":
        grad = (dy.t() @ h) * w + db[:, None] * b
        return (grad + s["acc"].double() if case["accumulate"] else grad), db
    rstd = s["rstd"].double()
    # Rows of the norm's Jacobian: r (I - 1 1^T / K - h h^T / K).
    dh = dy * w
    along_one = torch.mv(dh, torch.ones(hidden, dtype=torch.float64, device="cuda")) / hidden
    along_h = torch.linalg.vecdot(dh, h, dim=1) / hidden
    dw = torch.linalg.vecdot(dy, h, dim=0)
    dh.sub_(along_one[:, None]).sub_(along_h[:, None] * h).mul_(rstd[:, None])
    return dh, dw, db
