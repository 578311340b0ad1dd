"""The operators around the frozen-base linear layer that a transformer block's
projections need next to the product itself, as measured cases:

  forward     Z = X W'^T + s (X A) B + bias,  Y = act(Z) * mul + residual
              (api.qlora_linear_act_fwd; optionally Z kept, in 16 or in 8 bits)
  checkpoint  an activation held in 8 bits: per 64 consecutive values (row-major)
              one fp32 scale d = fl32(max|x| / 127) and codes
              q = round(x * fl32(127 / max|x|)), half to even; it stands for q d
              (api.act8_quantize, api.act8_dequantize)
  backward    dZ = dY * mul * act'(Z), dmul = dY * act(Z), dbias = sum_t dZ,
              dX = dZ W' + s (dZ B^T) A^T + dx_add, dA = s X^T (dZ B^T),
              dB = s (X A)^T dZ, with X, Z and mul read from 8-bit checkpoints
              (api.qlora_linear_act_bwd)

W' [N, K] is the frozen weight in 4-bit NormalFloat with double quantization (or
with one fp32 absmax per 64 weights, storage "sq"), rounded to the compute type;
A [K, r] and B [r, N] are the adapter.  `run` computes one case, in plain torch
operations or (`own`) through the framework's entry points; `exact` is the same
from the definitions in 64 bits.
"""
import math
from statistics import NormalDist

import torch

own = False

BLOCK = 64                       # weights per NF4 block, values per checkpoint block
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def _case(name, op, T, N, K, r, dtype="bf16", act="none", bias=False, mul=False, residual=False, save="none",
          storage="dq"):
    return dict(name=name, op=op, T=T, N=N, K=K, r=r, dtype=dtype, act=act, bias=bias, mul=mul, residual=residual,
                save=save, storage=storage)


def listed():
    return [
        # one new token through the gate projection of a 7B block: SiLU, times the up projection's output
        _case("fwd 1 token gate", "fwd", 1, 11008, 4096, 64, act="silu", mul=True),
        # a batch of seven sequences' next tokens through its down projection, added to the residual stream
        _case("fwd 7 tokens down", "fwd", 7, 4096, 11008, 64, residual=True),
        # a short prompt through a biased projection without an adapter, in fp16
        _case("fwd 61 tokens gelu", "fwd", 61, 4096, 4096, 0, dtype="fp16", act="gelu", bias=True, residual=True),
        # a mid-size prompt of odd length, the pre-activation kept for a backward pass
        _case("fwd 777 tokens gelu_tanh", "fwd", 777, 4096, 4096, 16, act="gelu_tanh", bias=True, residual=True,
              save="z"),
        # the gate projection of a 65B block in a training forward
        _case("fwd 2048 tokens 65B gate", "fwd", 2048, 22016, 8192, 64, act="silu", mul=True),
        # the checkpoint of one small input, written and read back
        _case("checkpoint 16 x 4096", "checkpoint", 16, 4096, 0, 0),
        # an odd number of values in fp16: the last block is a partial one
        _case("checkpoint 1531 x 4099", "checkpoint", 1531, 4099, 0, 0, dtype="fp16"),
        # the hidden activation of a 65B block at 2048 tokens
        _case("checkpoint 2048 x 22016", "checkpoint", 2048, 22016, 0, 0),
        # a short odd micro-batch through a biased fp16 projection
        _case("bwd 333 tokens gelu", "bwd", 333, 4096, 4096, 16, dtype="fp16", act="gelu", bias=True),
        # the gate projection of a 7B block in training: input, pre-activation and up output from checkpoints,
        # the up projection's input gradient added in
        _case("bwd 2048 tokens gate", "bwd", 2048, 11008, 4096, 64, act="silu", mul=True, residual=True),
        # its down projection at the 7B workload's 4096 tokens
        _case("bwd 4096 tokens down", "bwd", 4096, 4096, 11008, 64),
        # a whole training step of a biased projection: forward that keeps Z in 8 bits, checkpoint of X, backward
        _case("step 1000 tokens gelu", "step", 1000, 11008, 4096, 24, act="gelu", bias=True, save="z8"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("fwd", "fwd", "checkpoint", "bwd", "step"))
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    if op == "checkpoint":
        T, C = spread(1, 4096), spread(1, 22016)
        return {k: v for k, v in _case("", op, min(T, (2048 * 22016) // C), C, 0, 0, dtype=dtype).items() if k != "name"}
    T, N, K = spread(1, 4096), BLOCK * spread(1, 344), BLOCK * spread(1, 344)
    # at most the listed work of its kind: 2048 x 22016 x 8192 forward, 4096 x 4096 x 11008 backward
    T = max(1, min(T, (2048 * 22016 * 8192 if op == "fwd" else 4096 * 4096 * 11008 // 2) // (N * K)))
    act = rng.choice(ACTS)
    case = _case("", op, T, N, K, rng.choice((0, 8, 16, 24, 64, 128)), dtype=dtype, act=act,
                 bias=rng.random() < 0.5, mul=rng.random() < 0.4, residual=rng.random() < 0.5,
                 save={"fwd": rng.choice(("none", "z")), "bwd": "none", "step": "z8"}[op],
                 storage="sq" if dtype == "bf16" and rng.random() < 0.2 else "dq")
    return {k: v for k, v in case.items() if k != "name"}


# ------------------------------------------------------------------ what a program has in hand

def _dtype(case):
    return torch.float16 if case["dtype"] == "fp16" else torch.bfloat16


def _checkpoint(x):
    """(codes int8, scales fp32) of x, blocks of 64 consecutive values, the last one padded with zeros."""
    v = x.reshape(-1).float()
    v = torch.nn.functional.pad(v, (0, -v.numel() % BLOCK)).view(-1, BLOCK)
    top = v.abs().amax(1, keepdim=True)
    inv = torch.where(top > 0, 127.0 / top, torch.zeros_like(top))
    return torch.round(v * inv).to(torch.int8).view(-1)[:x.numel()].contiguous(), (top / 127.0).view(-1)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = _dtype(case)
    T, N, K, r, op = case["T"], case["N"], case["K"], case["r"], case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(dt)

    s = {"case": case, "dtype": dt}
    if op == "checkpoint":
        # activations: normal, with one channel in 64 thirty times as large
        x = torch.randn((T, N), generator=g, device=dev, dtype=torch.float32)
        x[:, ::64] *= 30.0
        s["x"] = x.to(dt)
        return s
    # the frozen weight: codes of normal weights are about equally likely; block absmax 0.03 to 0.08
    s["codes"] = torch.randint(0, 256, (N * K // 2,), generator=g, device=dev, dtype=torch.uint8)
    if case["storage"] == "sq":
        s["absmax"] = torch.rand((N * K // BLOCK,), generator=g, device=dev, dtype=torch.float32).mul_(0.05).add_(0.03)
    else:
        s["absmax_fp8"] = torch.randint(0x70, 0x7F, (N * K // BLOCK,), generator=g, device=dev, dtype=torch.uint8)
        s["superscale"] = torch.rand((-(-N * K // (BLOCK * 256)),), generator=g, device=dev,
                                     dtype=torch.float32).mul_(0.05).add_(0.03).div_(448.0)
    x = normal(T, K)
    s["a"] = normal(K, r, std=0.01) if r else None
    s["b"] = normal(r, N, std=0.01) if r else None
    s["bias"] = normal(N, std=0.5) if case["bias"] else None
    s["scaling"] = 16.0 / r if r else 1.0
    s["mul"] = normal(T, N) if case["mul"] else None
    s["x"] = x
    if op in ("fwd", "step"):
        s["residual"] = normal(T, N) if case["residual"] else None
    if op in ("bwd", "step"):
        s["dy"] = normal(T, N)
        s["dx_add"] = normal(T, K) if case["residual"] and op == "bwd" else None
    if op == "bwd":
        # the forward left checkpoints of X, Z and mul
        s["x8"] = _checkpoint(x)
        s["z8"] = _checkpoint(normal(T, N, std=1.5)) if case["act"] != "none" or case["mul"] else None
        s["mul8"] = _checkpoint(s["mul"]) if case["mul"] else None
        s["x"] = s["mul"] = None
    return s


# ------------------------------------------------------------------ the plain form

def _codebook():
    nd, d = NormalDist(), 0.5 * ((1 - 1 / 30) + (1 - 1 / 32))
    z = nd.inv_cdf(d)
    return ([-nd.inv_cdf(0.5 + j * (d - 0.5) / 7) / z for j in range(7, 0, -1)] + [0.0] +
            [nd.inv_cdf(0.5 + j * (d - 0.5) / 8) / z for j in range(1, 9)])


CODEBOOK = _codebook()


def _plain_weight(s):
    """W' [N, K] in fp32: codeword times block constant, rounded to the compute type."""
    case = s["case"]
    cb = torch.tensor(CODEBOOK, dtype=torch.float32, device=s["codes"].device)
    c = s["codes"]
    q = cb[torch.stack((c >> 4, c & 15), 1).int()].view(-1, BLOCK)
    if "absmax" in s:
        c1 = s["absmax"]
    else:
        c1 = s["absmax_fp8"].view(torch.float8_e4m3fn).float() * s["superscale"].repeat_interleave(256)[:q.shape[0]]
    return (q * c1[:, None]).to(s["dtype"]).float().view(case["N"], case["K"])


def _plain_act(z, act):
    """(act(z), act'(z))"""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, 0.0), (z > 0).float()
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        p = 0.5 * torch.erfc(z * -math.sqrt(0.5))
        return z * p, p + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    p = 0.5 * (1.0 + torch.tanh(c * (z + 0.044715 * z * z * z)))
    return z * p, p + z * p * (1.0 - p) * (2.0 * c) * (1.0 + 3.0 * 0.044715 * z * z)


def _plain_value(ck, shape):
    """What a checkpoint stands for, in fp32."""
    codes, scale = ck
    return (codes.float() * scale.repeat_interleave(BLOCK)[:codes.numel()]).view(shape)


def _plain_fwd(s, w):
    x = s["x"].float()
    z = x @ w.t()
    if s["a"] is not None:
        z = z + s["scaling"] * ((x @ s["a"].float()) @ s["b"].float())
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _plain_act(z, s["case"]["act"])[0]
    if s["mul"] is not None:
        y = y * s["mul"].float()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["dtype"]), z.to(s["dtype"])


def _plain_bwd(s, w, x8, z8, mul):
    case, dt = s["case"], s["dtype"]
    T, N, K = case["T"], case["N"], case["K"]
    dy, out = s["dy"].float(), {}
    dz = dy
    if z8 is not None:
        h, dh = _plain_act(_plain_value(z8, (T, N)), case["act"])
        if mul is not None:
            out["dmul"] = (dy * h).to(dt)
            dz = dy * mul
        dz = dz * dh
    dx = dz @ w
    if s["a"] is not None:
        x, a, b = _plain_value(x8, (T, K)).to(dt).float(), s["a"].float(), s["b"].float()
        g = s["scaling"] * (dz @ b.t())
        dx = dx + g @ a.t()
        out["da"] = (x.t() @ g).to(dt)
        out["db"] = (s["scaling"] * ((x @ a).t() @ dz)).to(dt)
    if s["dx_add"] is not None:
        dx = dx + s["dx_add"].float()
    out["dx"] = dx.to(dt)
    if case["bias"]:
        out["dbias"] = dz.sum(0).to(dt)
    return out


def _run_plain(s):
    case = s["case"]
    if case["op"] == "checkpoint":
        return _plain_value(_checkpoint(s["x"]), s["x"].shape).to(s["dtype"])
    w = _plain_weight(s)
    if case["op"] == "fwd":
        y, z = _plain_fwd(s, w)
        return {"y": y, "z": z} if case["save"] == "z" else {"y": y}
    if case["op"] == "bwd":
        mul = _plain_value(s["mul8"], (case["T"], case["N"])) if case["mul"] else None
        return _plain_bwd(s, w, s["x8"], s["z8"], mul)
    y, z = _plain_fwd(s, w)
    mul = s["mul"].float() if case["mul"] else None
    needs_z = case["act"] != "none" or case["mul"]
    return {"y": y, **_plain_bwd(s, w, _checkpoint(s["x"]), _checkpoint(z) if needs_z else None, mul)}


# ------------------------------------------------------------------ the framework's entry points

def _own_bwd(api, s, qw, x8, z8, mul):
    case = s["case"]
    g = api.qlora_linear_act_bwd(s["dy"], qw, s["a"], s["b"], s["scaling"], act=case["act"], z=z8, mul=mul,
                                 x=x8 if case["r"] else None, lora_grads=case["r"] > 0, bias_grad=case["bias"],
                                 dx_add=s["dx_add"])
    out = {"dx": g.dx, "dmul": g.d_mul, "da": g.d_lora_a, "db": g.d_lora_b, "dbias": g.d_bias}
    return {k: v for k, v in out.items() if v is not None}


def _run_own(s):
    from qlora_linear_layers_amd import api
    case = s["case"]
    if case["op"] == "checkpoint":
        return api.act8_dequantize(api.act8_quantize(s["x"]), dtype=s["dtype"])
    T, N, K = case["T"], case["N"], case["K"]
    if "absmax" in s:
        qw = api.NF4WeightSQ(s["codes"], s["absmax"], N, K)
    else:
        qw = api.NF4Weight(s["codes"], s["absmax_fp8"], s["superscale"], N, K)
    if case["op"] == "bwd":
        x8, z8, mul8 = (api.Act8(*s[k], shape) if s[k] is not None else None
                        for k, shape in (("x8", (T, K)), ("z8", (T, N)), ("mul8", (T, N))))
        return _own_bwd(api, s, qw, x8, z8, mul8)
    needs_z = case["act"] != "none" or case["mul"]
    save = case["save"] if case["op"] == "fwd" else ("z8" if needs_z else "none")
    got = api.qlora_linear_act_fwd(s["x"], qw, s["a"], s["b"], s["scaling"], bias=s["bias"], act=case["act"],
                                   mul=s["mul"], residual=s["residual"], save=None if save == "none" else save)
    y, z = got if save != "none" else (got, None)
    if case["op"] == "fwd":
        return {"y": y, "z": z} if save == "z" else {"y": y}
    x8 = api.act8_quantize(s["x"]) if case["r"] else None
    return {"y": y, **_own_bwd(api, s, qw, x8, z, s["mul"])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    T, N, K, r, op = case["T"], case["N"], case["K"], case["r"], case["op"]
    ck = lambda n: n + 4 * -(-n // BLOCK)                      # bytes of a checkpoint of n values
    if op == "checkpoint":
        n = T * N
        return {"bytes": 4 * n + 2 * ck(n), "flops": 4 * n}
    weight = N * K // 2 + (N * K // 16 if case["storage"] == "sq" else N * K // 64 + 4 * -(-N * K // 16384))
    needs_z = case["act"] != "none" or case["mul"]
    adapter = 2 * r * (K + N)
    base = weight + adapter + 2 * N * case["bias"]
    fwd_flops = 2 * T * N * K + 2 * T * r * (K + N)
    # G = dZ B^T and its product with A^T; X A, dA and dB
    bwd_flops = 2 * T * N * K + 2 * T * r * (N + K) + 2 * T * r * (2 * K + N)
    y_bytes = 2 * T * N * (1 + case["residual"] + case["mul"])
    # gradients written (dX, dA, dB, dbias, dmul); dY and the gradient to add read
    grads = 2 * T * K + adapter + 2 * N * case["bias"] + 2 * T * N * (1 + case["mul"])
    if op == "fwd":
        return {"bytes": base + 2 * T * K + y_bytes + 2 * T * N * (case["save"] == "z"), "flops": fwd_flops}
    if op == "bwd":
        read = (ck(T * K) if r else 0) + (ck(T * N) if needs_z else 0) + (ck(T * N) if case["mul"] else 0)
        return {"bytes": base - 2 * N * case["bias"] + read + 2 * T * K * case["residual"] + grads, "flops": bwd_flops}
    return {"bytes": base + 2 * T * K + y_bytes + grads, "flops": fwd_flops + bwd_flops}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_checkpoint(x):
    """The value of every element's code, in 64 bits, of a tensor of 16-bit values."""
    flat = x.reshape(-1).double()
    n = flat.numel()
    blk = torch.arange(n, device=flat.device) // BLOCK
    top = torch.zeros((-(-n // BLOCK),), dtype=torch.float64, device=flat.device)
    top = top.scatter_reduce(0, blk, flat.abs(), "amax")[blk]
    unit = top / 127.0
    return torch.where(top > 0, torch.round(flat / torch.where(top > 0, unit, 1.0)) * unit, 0.0).view(x.shape)


def _exact_weight(s):
    """The stored weight's 16-bit values: the block constant and the product are each rounded to fp32."""
    n = s["codes"].numel() * 2
    level = torch.tensor(CODEBOOK, dtype=torch.float64, device=s["codes"].device).float().double()
    w = torch.empty(n, dtype=torch.float64, device=s["codes"].device)
    w[0::2] = level[(s["codes"] // 16).long()]
    w[1::2] = level[(s["codes"] % 16).long()]
    if "absmax" in s:
        c1 = s["absmax"].double()
    else:
        code = s["absmax_fp8"].double()                        # all codes here are normal: 1.mmm 2^(e - 7)
        e = torch.floor(code / 8)
        group = torch.arange(code.numel(), device=code.device) // 256
        c1 = ((1.0 + (code - 8 * e) / 8) * torch.exp2(e - 7) * s["superscale"].double()[group]).float().double()
    w = w.view(-1, BLOCK).mul_(c1.view(-1, 1)).float().to(s["dtype"]).double()
    return w.view(s["case"]["N"], s["case"]["K"])


def _exact_act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))


def _exact_slope(z, act):
    """act'(z), by differentiating act itself."""
    z = z.detach().requires_grad_(True)
    with torch.enable_grad():
        return torch.autograd.grad(_exact_act(z, act).sum(), z)[0]


def _exact_bwd(s, w, x, z, mul):
    case, out = s["case"], {}
    dz = s["dy"].double()
    if z is not None:
        if mul is not None:
            out["dmul"] = dz * _exact_act(z, case["act"])
            dz = dz * mul
        dz = dz * _exact_slope(z, case["act"])
    out["dx"] = torch.mm(dz, w)
    if s["a"] is not None:
        x, a, b, sc = x.to(s["dtype"]).double(), s["a"].double(), s["b"].double(), s["scaling"]
        dzb = torch.mm(dz, b.t())
        out["dx"] += sc * torch.mm(dzb, a.t())
        out["da"] = sc * torch.mm(x.t(), dzb)
        out["db"] = sc * torch.mm(torch.mm(x, a).t(), dz)
    if s["dx_add"] is not None:
        out["dx"] += s["dx_add"].double()
    if case["bias"]:
        out["dbias"] = dz.sum(0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "checkpoint":
        return _exact_checkpoint(s["x"])
    w = _exact_weight(s)
    if case["op"] == "bwd":
        value = lambda ck, cols: ((ck[0].double().view(-1, BLOCK) * ck[1].double().view(-1, 1))
                                  .view(case["T"], cols) if ck is not None else None)
        return _exact_bwd(s, w, value(s["x8"], case["K"]), value(s["z8"], case["N"]), value(s["mul8"], case["N"]))
    x = s["x"].double()
    z = torch.mm(x, w.t())
    if s["a"] is not None:
        z += s["scaling"] * torch.mm(torch.mm(x, s["a"].double()), s["b"].double())
    if s["bias"] is not None:
        z += s["bias"].double()
    mul = s["mul"].double() if s["mul"] is not None else None
    y = _exact_act(z, case["act"])
    if mul is not None:
        y = y * mul
    if s["residual"] is not None:
        y = y + s["residual"].double()
    if case["op"] == "fwd":
        return {"y": y, "z": z} if case["save"] == "z" else {"y": y}
    needs_z = case["act"] != "none" or case["mul"]
    kept = _exact_checkpoint(z.to(s["dtype"])) if needs_z else None      # the checkpoint is of the 16-bit Z
    return {"y": y, **_exact_bwd(s, w, _exact_checkpoint(s["x"]), kept, mul)}
