"""The norm in front of a transformer block, rows in 8 bits, and the 8-bit integer
product that serves a merged layer, as measured cases:

  norm      h = x + residual (rounded to the 16-bit type; h = x without one),
            y = h (mean(h^2) + eps)^(-1/2) w, in 16 bits or as 8-bit rows
            (api.rmsnorm_fwd)
  norm_bwd  with n = h (mean(h^2) + eps)^(-1/2), g = dy w:
            dx = (mean(h^2) + eps)^(-1/2) (g - n mean(g n)) + dx_add, dw = sum_t dy n
            (api.rmsnorm_bwd)
  rows8     a matrix held in 8 bits with one scale per row: c = max|row|,
            d = fl32(c / 127), codes q = round(x * fl32(127 / c)), half to even; it
            stands for q d (api.rows8_quantize, api.rows8_dequantize).  Rows are
            tokens of an activation or output channels of a weight
  linear8   y = act(sum_k xq wq * dx dw + bias) * mul + residual from the 8-bit
            rows of X [T, K] and W [N, K] (api.int8_linear_fwd)

Codes are stored with rows padded by zeros to a multiple of 128.  `run` computes one
case, in plain torch operations or (`own`) through the framework's entry points;
`exact` is the same from the definitions in 64 bits.
"""
import math

import torch

own = False

PITCH = 128                      # a row of codes takes a multiple of this many bytes
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def _case(name, op, T, N, K, dtype="bf16", residual=False, quantize=False, w32=False, eps=1e-6, act="none", bias=False,
          mul=False):
    """T rows of K values; N output channels of a product."""
    return dict(name=name, op=op, T=T, N=N, K=K, dtype=dtype, residual=residual, quantize=quantize, w32=w32, eps=eps,
                act=act, bias=bias, mul=mul)


def listed():
    return [
        # one new token's hidden state in front of a 7B block
        _case("norm 1 token", "norm", 1, 0, 4096, residual=True),
        # an odd row length in fp16, the first norm of a model (nothing to add), fp32 weights
        _case("norm 1531 x 4099", "norm", 1531, 0, 4099, dtype="fp16", w32=True, eps=1e-5),
        # a 65B prompt's hidden states, written as the 8-bit rows that the next product reads
        _case("norm 2048 x 8192 to 8 bits", "norm", 2048, 0, 8192, residual=True, quantize=True),
        # a short odd micro-batch in training
        _case("norm_bwd 333 x 4096", "norm_bwd", 333, 0, 4096, dtype="fp16"),
        # a 65B training batch: fp32 norm weights, the residual path's gradient added
        _case("norm_bwd 4096 x 8192", "norm_bwd", 4096, 0, 8192, residual=True, w32=True),
        # seven tokens' hidden activation in front of a 7B down projection
        _case("rows8 7 x 11008", "rows8", 7, 0, 11008),
        # the hidden activation of a 65B block at 2048 tokens
        _case("rows8 2048 x 22016", "rows8", 2048, 0, 22016),
        # one new token through the gate projection of a 7B block: SiLU, times the up projection's output
        _case("linear8 1 token gate", "linear8", 1, 11008, 4096, act="silu", mul=True),
        # a batch of seven sequences' next tokens through its down projection, added to the residual stream
        _case("linear8 7 tokens down", "linear8", 7, 4096, 11008, residual=True),
        # a short prompt through a biased fp16 projection of odd sizes
        _case("linear8 61 tokens 4099 to 4097", "linear8", 61, 4097, 4099, dtype="fp16", act="gelu", bias=True),
        # a mid-size prompt of odd length
        _case("linear8 777 tokens", "linear8", 777, 4096, 4096, act="gelu_tanh", bias=True, residual=True),
        # the gate projection of a 65B block at 2048 tokens
        _case("linear8 2048 tokens 65B gate", "linear8", 2048, 22016, 8192, act="silu", mul=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("norm", "norm", "norm_bwd", "rows8", "linear8", "linear8", "linear8"))
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    T, K = spread(1, 4096), spread(8, 22016)
    # row lengths of models are multiples of 64; one in four here is any number
    K = K if rng.random() < 0.25 else max(64, K // 64 * 64)
    if op == "linear8":
        N = spread(1, 22016)
        N = N if rng.random() < 0.25 else max(64, N // 64 * 64)
        T = max(1, min(T, (2048 * 22016 * 8192) // (N * K)))
        case = _case("", op, T, N, K, dtype=dtype, act=rng.choice(ACTS), bias=rng.random() < 0.5,
                     mul=rng.random() < 0.4, residual=rng.random() < 0.5)
    else:
        T = max(1, min(T, (4096 * 8192) // K))
        case = _case("", op, T, 0, K, dtype=dtype, residual=op != "rows8" and rng.random() < 0.6,
                     quantize=op == "norm" and rng.random() < 0.5, w32=op != "rows8" and rng.random() < 0.4,
                     eps=rng.choice((1e-6, 1e-5)))
    return {k: v for k, v in case.items() if k != "name"}


# ------------------------------------------------------------------ what a program has in hand

def _dtype(case):
    return torch.float16 if case["dtype"] == "fp16" else torch.bfloat16


def _rows8(x):
    """(codes int8 [R, K], scale fp32 [R, 1]) of a matrix in fp32."""
    top = x.abs().amax(1, keepdim=True)
    inv = torch.where(top > 0, 127.0 / top, torch.zeros_like(top))
    return torch.round(x * inv).to(torch.int8), top / 127.0


def _stored(x):
    """Codes padded to whole pitches, and the scales, of a matrix in fp32."""
    codes, scale = _rows8(x)
    return torch.nn.functional.pad(codes, (0, -codes.shape[1] % PITCH)).contiguous(), scale.view(-1)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = _dtype(case)
    T, N, K, op = case["T"], case["N"], case["K"], case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(std)

    def hidden(rows, cols):
        # activations: normal, with one channel in 64 much larger, as hidden states have
        x = normal(rows, cols)
        x[:, ::64] *= 10.0
        return x

    s = {"case": case, "dtype": dt}
    if op in ("norm", "norm_bwd"):
        s["weight"] = normal(K, std=0.2).add_(1.0).to(torch.float32 if case["w32"] else dt)
        s["x"] = hidden(T, K).to(dt)
        if op == "norm":
            s["residual"] = hidden(T, K).to(dt) if case["residual"] else None
        else:
            s["dy"] = normal(T, K).to(dt)
            s["dx_add"] = normal(T, K).to(dt) if case["residual"] else None
    elif op == "rows8":
        s["x"] = hidden(T, K).to(dt)
    else:
        s["x_codes"], s["x_scale"] = _stored(hidden(T, K).to(dt).float())
        s["w_codes"], s["w_scale"] = _stored(normal(N, K, std=K ** -0.5).to(dt).float())
        s["bias"] = normal(N, std=0.5).to(dt) if case["bias"] else None
        s["mul"] = normal(T, N).to(dt) if case["mul"] else None
        s["residual"] = normal(T, N).to(dt) if case["residual"] else None
    return s


# ------------------------------------------------------------------ the plain form

def _plain_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return z * 0.5 * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_norm(s):
    case, dt = s["case"], s["dtype"]
    h, out = s["x"], {}
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(dt)
        out["h"] = h
    h = h.float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + case["eps"]) * s["weight"].float()
    if case["quantize"]:
        codes, scale = _rows8(y)
        y = codes.float() * scale
    out["y"] = y.to(dt)
    return out


def _plain_norm_bwd(s):
    case, dt = s["case"], s["dtype"]
    h, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + case["eps"])
    n = h * r
    g = dy * s["weight"].float()
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    if s["dx_add"] is not None:
        dx = dx + s["dx_add"].float()
    return {"dx": dx.to(dt), "dw": (dy * n).sum(0).to(s["weight"].dtype)}


def _plain_linear8(s):
    case, dt, K = s["case"], s["dtype"], s["case"]["K"]
    z = s["x_codes"][:, :K].float() @ s["w_codes"][:, :K].float().t()
    z = z * (s["x_scale"][:, None] * s["w_scale"][None, :])
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _plain_act(z, case["act"])
    if s["mul"] is not None:
        y = y * s["mul"].float()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(dt)}


def _run_plain(s):
    op = s["case"]["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    if op == "rows8":
        codes, scale = _rows8(s["x"].float())
        return (codes.float() * scale).to(s["dtype"])
    return _plain_linear8(s)


# ------------------------------------------------------------------ the framework's entry points

def _run_own(s):
    from qlora_linear_layers_amd import api
    case, dt = s["case"], s["dtype"]
    op = case["op"]
    if op == "norm":
        got = api.rmsnorm_fwd(s["x"], s["weight"], case["eps"], residual=s["residual"], quantize=case["quantize"])
        y, h = got if s["residual"] is not None else (got, None)
        if case["quantize"]:
            y = api.rows8_dequantize(y, dtype=dt)
        return {"y": y} if h is None else {"y": y, "h": h}
    if op == "norm_bwd":
        g = api.rmsnorm_bwd(s["dy"], s["x"], s["weight"], case["eps"], dx_add=s["dx_add"])
        return {"dx": g.dx, "dw": g.d_weight}
    if op == "rows8":
        return api.rows8_dequantize(api.rows8_quantize(s["x"]), dtype=dt)
    x8 = api.Rows8(s["x_codes"], s["x_scale"], (case["T"], case["K"]))
    w8 = api.Rows8(s["w_codes"], s["w_scale"], (case["N"], case["K"]))
    return {"y": api.int8_linear_fwd(x8, w8, dtype=dt, bias=s["bias"], act=case["act"], mul=s["mul"],
                                     residual=s["residual"])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    T, N, K, op = case["T"], case["N"], case["K"], case["op"]
    rows8 = lambda rows: rows * (K + 4)                        # bytes of 8-bit rows
    weight = K * (4 if case["w32"] else 2)
    if op == "norm":
        moved = 2 * T * K * (2 + 2 * case["residual"])         # x and y; residual and h
        if case["quantize"]:                                   # the rows written, and read back into y
            moved += 2 * rows8(T)
        return {"bytes": moved + weight, "flops": T * K * (4 + case["residual"] + 3 * case["quantize"])}
    if op == "norm_bwd":
        return {"bytes": 2 * T * K * (3 + case["residual"]) + 2 * weight, "flops": T * K * (11 + case["residual"])}
    if op == "rows8":
        return {"bytes": 4 * T * K + 2 * rows8(T), "flops": 4 * T * K}
    return {"bytes": rows8(T) + rows8(N) + 2 * N * case["bias"] + 2 * T * N * (1 + case["mul"] + case["residual"]),
            "flops": 2 * T * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rows8(x):
    """What the 8-bit rows of a matrix in 64 bits stand for."""
    unit = x.abs().max(dim=1, keepdim=True).values / 127.0
    return torch.where(unit > 0, torch.round(x / torch.where(unit > 0, unit, 1.0)) * unit, 0.0)


def _exact_act(z, act):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _exact_normed(h, weight, eps):
    return h / torch.sqrt(h.square().sum(1, keepdim=True) / h.shape[1] + eps) * weight


def exact(case, seed):
    s = prepare(case, seed)
    op, K = case["op"], case["K"]
    if op == "norm":
        h, out = s["x"].double(), {}
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["dtype"]).double()       # the stream is kept in 16 bits
            out["h"] = h
        y = _exact_normed(h, s["weight"].double(), case["eps"])
        out["y"] = _exact_rows8(y) if case["quantize"] else y
        return out
    if op == "norm_bwd":
        # by differentiating the norm itself
        h, w = s["x"].double().requires_grad_(True), s["weight"].double().requires_grad_(True)
        with torch.enable_grad():
            dx, dw = torch.autograd.grad(_exact_normed(h, w, case["eps"]), (h, w), s["dy"].double())
        return {"dx": dx if s["dx_add"] is None else dx + s["dx_add"].double(), "dw": dw}
    if op == "rows8":
        return _exact_rows8(s["x"].double())
    x = s["x_codes"][:, :K].double() * s["x_scale"].double()[:, None]
    w = s["w_codes"][:, :K].double() * s["w_scale"].double()[:, None]
    z = torch.mm(x, w.t())
    if s["bias"] is not None:
        z += s["bias"].double()
    y = _exact_act(z, case["act"])
    if s["mul"] is not None:
        y = y * s["mul"].double()
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return {"y": y}
