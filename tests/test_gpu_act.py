"""The layer's epilogue forward, the 8-bit activation checkpoint and the backward
from saved activations on the GPU, against the fp64 oracle.

Tolerances.  u is the unit roundoff of the 16-bit type (2^-8 bf16, 2^-11 fp16).
Checkpoints (codes, scales, values) are bit-exact.  Every other output is a sum
accumulated in fp32 and rounded once.  The products of the backward take dZ
rounded to 16 bits, in the oracle too, but an fp32 dZ next to a rounding
boundary can go the other way than the fp64 one: noise far below u/sqrt(3) of
the output's rms.  So the relative 2-norm error is below u, and no element is
off by more than u |y| + 4 u rms."""
import numpy as np
import pytest
import torch

import oracle
from qlora_linear_layers_amd import api
from helpers import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, ref, what):
    u, g, ref = U[got.dtype], f64(got), np.asarray(ref)
    assert g.shape == ref.shape, what
    assert np.isfinite(g).all(), what
    rms = float(np.sqrt(np.mean(ref * ref)))
    err = np.abs(g - ref)
    rel = float(np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-300))
    over = float(np.max(err - (u * np.abs(ref) + 4 * u * rms)))
    say(f"  {what}: rel2={rel / u:.3f} u, worst excess {over:.2e}")
    # a handful of values can all round badly: the 2-norm bound needs some to average over
    assert over <= 0 and (g.size < 256 or rel <= u), what


class Case:
    def __init__(self, T, N, K, r, dtype="bf16", storage="dq", seed=0, s=0.5):
        g = torch.Generator().manual_seed(1000 * T + 10 * N + K + r + seed)
        self.T, self.N, self.K, self.r, self.s, self.dt = T, N, K, r, s, DT[dtype]
        n = lambda *sh, std=1.0: (torch.randn(sh, generator=g) * std).to(self.dt).cuda()
        w = n(N, K, std=2.0 / K ** 0.5)
        self.qw = api.nf4_quantize(w) if storage == "sq" else api.nf4_quantize_dq(w)
        self.wd = f64(api.nf4_dequantize(self.qw) if storage == "sq" else
                      api.nf4_dequantize_dq(self.qw, dtype=self.dt))
        self.x = n(T, K)
        self.a, self.b = (n(K, r, std=0.05), n(r, N, std=0.2)) if r else (None, None)
        self.bias, self.mul, self.res = n(N, std=0.5), n(T, N), n(T, N)
        self.z, self.dy, self.add = n(T, N, std=1.5), n(T, N), n(T, K)

    def ab64(self):
        return (f64(self.a), f64(self.b)) if self.r else (None, None)


# every route of the forward: decode (T <= 16; one and two columns per lane, one
# and two tokens per wave, ragged last column group), 16-token windows with an
# overlapping last one, split tiles, whole tiles with ragged edges in both directions
ROUTES = [(1, 64, 64, 0), (1, 192, 448, 16), (3, 320, 192, 8), (7, 192, 576, 72), (16, 320, 256, 24),
          (17, 192, 320, 16), (61, 256, 192, 0), (96, 128, 64, 8), (97, 320, 448, 24), (300, 448, 320, 16),
          (333, 1024, 2048, 64), (513, 4160, 128, 0)]


@pytest.mark.parametrize("T,N,K,r", ROUTES)
@pytest.mark.parametrize("act,bias,mul,res", [("silu", False, True, False), ("gelu", True, False, True),
                                              ("none", True, True, True)])
def test_forward_epilogue(T, N, K, r, act, bias, mul, res):
    say(f"[act fwd] T={T} N={N} K={K} r={r} {act} bias={bias} mul={mul} res={res}")
    c = Case(T, N, K, r)
    kw = dict(bias=c.bias if bias else None, act=act, mul=c.mul if mul else None, residual=c.res if res else None)
    y, z = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s, save="z", **kw)
    y2, z8 = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s, save="z8", **kw)
    y3 = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s, **kw)
    q = api.act8_quantize(z)
    torch.cuda.synchronize()
    ry, rz = oracle.act_fwd(f64(c.x), c.wd, *c.ab64(), c.s, f64(c.bias) if bias else None, act,
                            f64(c.mul) if mul else None, f64(c.res) if res else None)
    check(z, rz, "Z")
    check(y, ry, "Y")
    assert torch.equal(y, y2) and torch.equal(y, y3)
    # the saved checkpoint is that of the 16-bit Z, bit for bit
    assert torch.equal(z8.codes, q.codes) and torch.equal(z8.scale, q.scale)


@pytest.mark.parametrize("T", [2, 40, 300, 600])
@pytest.mark.parametrize("act", oracle.ACTS)
@pytest.mark.parametrize("dtype,storage", [("bf16", "dq"), ("bf16", "sq"), ("fp16", "dq")])
def test_forward_types(T, act, dtype, storage):
    say(f"[act fwd] T={T} {act} {dtype} {storage}")
    c = Case(T, 320, 192, 8, dtype, storage)
    y, z = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s, bias=c.bias, act=act, mul=c.mul, residual=c.res, save="z")
    torch.cuda.synchronize()
    ry, rz = oracle.act_fwd(f64(c.x), c.wd, *c.ab64(), c.s, f64(c.bias), act, f64(c.mul), f64(c.res))
    check(z, rz, "Z")
    check(y, ry, "Y")


@pytest.mark.parametrize("T", [1, 9, 33, 200, 700])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_empty_epilogue_is_the_plain_forward(T, dtype):
    say(f"[act fwd] empty epilogue T={T} {dtype}")
    c = Case(T, 448, 256, 16, dtype)
    y = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s)
    assert torch.equal(y.view(torch.int16), api.qlora_linear_fwd(c.x, c.qw, c.a, c.b, c.s).view(torch.int16))


@pytest.mark.parametrize("T", [5, 61, 300, 513])
def test_output_in_place_of_residual_or_mul(T):
    """y may be the buffer of residual or of mul, on every route (61: the windows overlap)."""
    say(f"[act fwd] in place T={T}")
    c = Case(T, 320, 192, 8)
    kw = dict(act="gelu_tanh", bias=c.bias)
    ref = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s, mul=c.mul, residual=c.res, **kw)
    for name in ("residual", "mul"):
        t = {"mul": c.mul.clone(), "residual": c.res.clone()}
        y = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s, out=t[name], **t, **kw)
        assert y is t[name] and torch.equal(y, ref), name


def test_large_and_extreme_preactivations():
    """Pre-activations from tiny to 1e30: no inf - inf or inf * 0 in any activation or slope."""
    N, K, T = 64, 64, 4
    w = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 1.0
    qw = api.nf4_quantize_dq(w)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    for t, v in enumerate((1e30, -1e30, 1e-30, -90.0)):
        x[t, 0] = v
    wd = f64(api.nf4_dequantize_dq(qw))
    for act in oracle.ACTS:
        say(f"[act] extreme {act}")
        y, z = api.qlora_linear_act_fwd(x, qw, act=act, save="z")
        with np.errstate(all="ignore"):
            ry = oracle.act(f64(x) @ wd.T, act)
        ry = np.where(np.abs(ry) < 1e-35, 0.0, ry)
        assert np.all(np.abs(f64(y) - ry) <= 2.0 ** -8 * np.abs(ry) + 1e-30), act
        g = api.qlora_linear_act_bwd(torch.ones_like(y), qw, act=act, z=z, bias_grad=True)
        assert torch.isfinite(g.dx).all() and torch.isfinite(g.d_bias).all(), act


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", [a for a in oracle.ACTS if a != "none"])
def test_slopes_over_the_range(act, dtype):
    """With one token d_bias is dY act'(Z) and d_mul dY act(Z), each rounded once.  Z covers the
    type's magnitudes in both signs; the fp32 terms of a slope (p, and z times an exponentially
    small factor) are good to a few 2^-24 of 1, or of the result where that is larger."""
    dt, N = DT[dtype], 1024
    top = 4.5 if dtype == "fp16" else 30.0
    m = torch.logspace(-6, top, N // 2 - 32, dtype=torch.float64)
    z = torch.cat([m, -m, torch.linspace(-12, 12, 63, dtype=torch.float64), torch.zeros(1, dtype=torch.float64)])
    z = z.to(dt).reshape(1, N).cuda()
    qw = api.nf4_quantize_dq(torch.ones(N, 64, dtype=dt, device="cuda"))
    one = torch.ones(1, N, dtype=dt, device="cuda")
    say(f"[act] slopes {act} {dtype}")
    g = api.qlora_linear_act_bwd(one, qw, act=act, z=z, mul=one, bias_grad=True)
    with np.errstate(all="ignore"):
        rd, rv = oracle.act_slope(f64(z), act)[0], oracle.act(f64(z), act)
    rd = np.where(np.isnan(rd), (f64(z)[0] > 0).astype(float), rd)      # 0 * inf in the fp64 tails of the tanh form
    u = U[dt]
    assert np.all(np.abs(f64(g.d_bias) - rd) <= u * np.abs(rd) + 2.0 ** -20)
    assert np.all(np.abs(f64(g.d_mul) - rv) <= u * np.abs(rv) + 2.0 ** -20)


@pytest.mark.parametrize("act", oracle.ACTS)
def test_nan_is_not_lost(act):
    """A NaN pre-activation is NaN in Y, Z and its checkpoint, and in the gradients that read it."""
    c = Case(3, 128, 64, 0)
    x = c.x.clone()
    x[1, 5] = float("nan")
    say(f"[act] nan {act}")
    y, z8 = api.qlora_linear_act_fwd(x, c.qw, act=act, mul=c.mul, save="z8")
    assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2]]).all()
    z = api.act8_dequantize(z8)
    assert torch.isnan(z[1]).all() and torch.isfinite(z[[0, 2]]).all()
    for saved in (z, z8):
        g = api.qlora_linear_act_bwd(c.dy, c.qw, act=act, z=saved, mul=c.mul)
        assert torch.isnan(g.d_mul[1]).all() and torch.isfinite(g.d_mul[[0, 2]]).all()
        assert torch.isfinite(g.dx[[0, 2]]).all()
        if act != "none":
            assert torch.isnan(g.dx[1]).all()


# ------------------------------------------------------------------ checkpoints

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", [(1,), (63,), (64,), (65,), (7, 9), (3, 64), (33, 1000), (129, 4099), (5, 3, 77)])
def test_checkpoint_bit_exact(shape, dtype):
    say(f"[act8] {shape} {dtype}")
    g = torch.Generator().manual_seed(7)
    x = torch.randn(shape, generator=g)
    x[..., ::17] *= 40.0
    x = x.to(DT[dtype]).cuda()
    n = x.numel()
    # guard values after every output
    pad = lambda k, d: torch.full((k + 64,), 77, dtype=d, device="cuda")
    codes, scale, val = pad(n, torch.int8), pad(-(-n // 64), torch.float32), pad(n, DT[dtype])
    a8 = api.Act8(codes[:n], scale[:-(-n // 64)], tuple(shape))
    api.act8_quantize(x, out=a8)
    v = api.act8_dequantize(a8, out=val[:n].view(shape))
    torch.cuda.synchronize()
    q, d = oracle.ck_quantize(f64(x))
    assert np.array_equal(a8.codes.cpu().numpy(), q)
    assert np.array_equal(a8.scale.cpu().numpy().view(np.uint32), d.view(np.uint32))
    ref = torch.from_numpy(oracle.ck_values(q, d)).to(DT[dtype]).view(shape)   # fp64 of an fp32 value: one rounding
    assert torch.equal(v.cpu(), ref)
    for t, k in ((codes, n), (scale, -(-n // 64)), (val, n)):
        assert torch.all(t[k:] == 77)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_checkpoint_edge_blocks(dtype):
    """All-zero, tiny, subnormal, largest, non-finite and half-way blocks."""
    dt = DT[dtype]
    top = float(torch.finfo(dt).max)
    tiny = 2.0 ** -133 if dtype == "bf16" else 2.0 ** -24
    x = torch.zeros((12, 64), dtype=dt)
    g = torch.Generator().manual_seed(3)
    r = torch.randn((12, 64), generator=g)
    x[1] = (r[1] * 2.0 ** -123).to(dt) if dtype == "bf16" else (r[1] * tiny * 4).to(dt)
    x[2] = (r[2] * 2.0 ** -119).to(dt)
    x[3, 5] = tiny
    x[4] = (r[4] / r[4].abs().max() * top).to(dt)
    x[5] = r[5].to(dt)
    x[5, 11] = float("inf")
    x[6] = r[6].to(dt)
    x[6, 63] = float("nan")
    x[7, 0] = float("-inf")
    x[8, :4] = torch.tensor([254.0, 127.0, 1.0, -3.0])
    x[9] = -0.0
    x[10, 17] = -top
    x[11] = r[11].to(dt)
    x = x.cuda()
    a8 = api.act8_quantize(x)
    v = api.act8_dequantize(a8, dtype=dt)
    torch.cuda.synchronize()
    q, d = oracle.ck_quantize(f64(x))
    assert np.array_equal(a8.codes.cpu().numpy(), q)
    got = a8.scale.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(d)) and np.array_equal(got[~np.isnan(d)], d[~np.isnan(d)])
    bad = torch.tensor([5, 6, 7])
    assert torch.isnan(v[bad]).all()
    ok = [i for i in range(12) if i not in (5, 6, 7)]
    ref = torch.from_numpy(oracle.ck_values(q, d)).to(dt).view(12, 64)
    assert torch.equal(v.cpu()[ok], ref[ok])


# ------------------------------------------------------------------ backward

def _saved(t, form):
    """(what the call gets, the fp64 values it stands for) of a saved activation."""
    if form == "8":
        a8 = api.act8_quantize(t)
        return a8, oracle.ck_values(a8.codes.cpu().numpy(), a8.scale.cpu().numpy()).reshape(t.shape)
    return t, f64(t)


def _backward(c, act, mul, form, bias=True, add=False, what=""):
    say(f"[act bwd] T={c.T} N={c.N} K={c.K} r={c.r} {act} mul={mul} saved as {form} bits {what}")
    needs_z = act != "none" or mul
    z, rz = _saved(c.z, form) if needs_z else (None, None)
    m, rm = _saved(c.mul, form) if mul else (None, None)
    x, _ = _saved(c.x, form) if c.r else (None, None)
    # X enters the products in 16 bits in either form
    rx = f64(api.act8_dequantize(x, dtype=c.dt)) if form == "8" and c.r else f64(c.x)
    g = api.qlora_linear_act_bwd(c.dy, c.qw, c.a, c.b, c.s, act=act, x=x, z=z, mul=m, lora_grads=c.r > 0,
                                 bias_grad=bias, dx_add=c.add if add else None)
    torch.cuda.synchronize()
    ref = oracle.act_bwd(f64(c.dy), c.wd, *c.ab64(), c.s, act, rx, rz, rm, f64(c.add) if add else None,
                         round16=lambda v: f64(torch.from_numpy(v).to(c.dt)))
    check(g.dx, ref["dx"], "dX")
    for name, key in (("d_bias", "dbias"), ("d_mul", "dmul"), ("d_lora_a", "da"), ("d_lora_b", "db")):
        got = getattr(g, name)
        asked = {"d_bias": bias, "d_mul": mul}.get(name, c.r > 0)
        assert (got is not None) == asked, name
        if asked:
            check(got, ref[key], name)
    return g


@pytest.mark.parametrize("T,N,K,r", [(1, 64, 64, 0), (1, 192, 128, 8), (17, 320, 448, 16), (130, 192, 4480, 24),
                                     (300, 448, 320, 72), (1000, 192, 192, 8), (513, 1024, 4096, 16)])
@pytest.mark.parametrize("act,mul", [("silu", True), ("gelu", False), ("none", False), ("none", True)])
@pytest.mark.parametrize("form", ["8", "16"])
def test_backward(T, N, K, r, act, mul, form):
    _backward(Case(T, N, K, r), act, mul, form, add=T % 2 == 1)


@pytest.mark.parametrize("act", oracle.ACTS)
@pytest.mark.parametrize("dtype,storage", [("bf16", "sq"), ("fp16", "dq")])
def test_backward_types(act, dtype, storage):
    c = Case(150, 256, 320, 16, dtype, storage)
    _backward(c, act, True, "8", add=True, what=f"{dtype} {storage}")
    _backward(c, act, False, "16", bias=False, what=f"{dtype} {storage}")


def test_backward_many_row_ranges():
    """More than 64 * 128 rows: the column sums' ranges grow."""
    _backward(Case(9001, 64, 64, 8), "relu", False, "8")


def test_backward_matches_the_plain_backward():
    """Without activation, mul and bias gradient the call is the plain backward: the same bits,
    with X in 16 bits or as the checkpoint of exactly representable values."""
    c = Case(300, 448, 320, 16)
    dx, da, db = api.qlora_linear_bwd_input(c.dy, c.qw, c.a, c.b, c.s, x=c.x, lora_grads=True)
    g = api.qlora_linear_act_bwd(c.dy, c.qw, c.a, c.b, c.s, x=c.x, lora_grads=True)
    assert torch.equal(g.dx, dx) and torch.equal(g.d_lora_a, da) and torch.equal(g.d_lora_b, db)
    a8 = api.act8_quantize(c.x)
    xq = api.act8_dequantize(a8)
    dx, da, db = api.qlora_linear_bwd_input(c.dy, c.qw, c.a, c.b, c.s, x=xq, lora_grads=True)
    g = api.qlora_linear_act_bwd(c.dy, c.qw, c.a, c.b, c.s, x=a8, lora_grads=True)
    assert torch.equal(g.dx, dx) and torch.equal(g.d_lora_a, da) and torch.equal(g.d_lora_b, db)


@pytest.mark.parametrize("T", [20, 300])
def test_dx_add_in_place(T):
    c = Case(T, 320, 448, 8)
    ref = api.qlora_linear_act_bwd(c.dy, c.qw, c.a, c.b, c.s, dx_add=c.add).dx
    acc = c.add.clone()
    g = api.qlora_linear_act_bwd(c.dy, c.qw, c.a, c.b, c.s, dx_add=acc, dx=acc)
    assert g.dx is acc and torch.equal(acc, ref)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(act):
    """<grad, v> from the kernels against central differences of the fp64 forward.  The 16-bit
    gradients' errors (at most u relative in the 2-norm) meet a random direction v, so the inner
    product is off by at most u |grad| |v| (Cauchy-Schwarz); the differences add less than 1e-6
    relative."""
    c = Case(40, 192, 128, 8)
    p = dict(x=f64(c.x), a=f64(c.a), b=f64(c.b), bias=f64(c.bias), mul=f64(c.mul))

    def loss(q):
        y, z = oracle.act_fwd(q["x"], c.wd, q["a"], q["b"], c.s, q["bias"], act, q["mul"])
        return float((y * f64(c.dy)).sum()), z
    # the Z of the oracle's own forward, kept in 16 bits: the slope's argument is off by u |Z|,
    # which |act''| <= 1.2 turns into at most 1.2 u |Z dY mul| in dZ
    z = torch.from_numpy(loss(p)[1]).to(c.dt).cuda()
    g = api.qlora_linear_act_bwd(c.dy, c.qw, c.a, c.b, c.s, act=act, x=c.x, z=z, mul=c.mul, lora_grads=True,
                                 bias_grad=True)
    rng = np.random.default_rng(2)
    u = U[c.dt]
    extra = 1.2 * u * float(np.linalg.norm(f64(z) * f64(c.dy) * f64(c.mul)))
    norm = lambda m: float(np.linalg.norm(m, 2))
    up = norm(c.wd) + c.s * norm(p["a"]) * norm(p["b"])
    gain = {"x": up, "bias": p["x"].shape[0] ** 0.5, "mul": 0.0, "a": c.s * norm(p["x"]) * norm(p["b"]),
            "b": c.s * norm(p["x"] @ p["a"])}
    for var, got in (("x", g.dx), ("a", g.d_lora_a), ("b", g.d_lora_b), ("bias", g.d_bias), ("mul", g.d_mul)):
        v = rng.standard_normal(p[var].shape)
        v /= np.linalg.norm(v)
        e = 1e-4
        d = (loss({**p, var: p[var] + e * v})[0] - loss({**p, var: p[var] - e * v})[0]) / (2 * e)
        h = float((f64(got) * v).sum())
        tol = u * float(np.linalg.norm(f64(got))) + gain[var] * extra + (1.2 * u * float(np.linalg.norm(
            f64(z) * f64(c.dy))) if var == "mul" else 0.0) + 1e-5
        say(f"  {act} d{var}: {h:.5f} against {d:.5f} (tol {tol:.5f})")
        assert abs(h - d) <= tol, var


def test_results_repeat_and_other_streams():
    """The same bits on every run, also on a stream of the caller's."""
    c = Case(300, 448, 320, 16)
    x8, z8 = api.act8_quantize(c.x), api.act8_quantize(c.z)

    def go():
        g = api.qlora_linear_act_bwd(c.dy, c.qw, c.a, c.b, c.s, act="gelu", x=x8, z=z8, lora_grads=True, bias_grad=True)
        y = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s, bias=c.bias, act="gelu", residual=c.res)
        return [g.dx, g.d_lora_a, g.d_lora_b, g.d_bias, y]
    ref = go()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        other = go()
    st.synchronize()
    for a, b, d in zip(ref, go(), other):
        assert torch.equal(a, b) and torch.equal(a, d)


def test_graph_replays():
    """A forward that keeps a checkpoint and its backward, recorded and replayed with new inputs."""
    c = Case(300, 448, 320, 16)
    z8 = api.act8_empty((c.T, c.N))
    x8 = api.act8_empty((c.T, c.K))
    y, dx = torch.empty_like(c.res), torch.empty_like(c.add)
    da, db, dbias = torch.empty_like(c.a), torch.empty_like(c.b), torch.empty_like(c.bias)
    wf = api.workspace_for(c.T, c.K, c.N, c.r, "cuda")
    wb = torch.empty(api.qlora_act_workspace_bytes_bwd(c.T, c.K, c.N, c.r), dtype=torch.uint8, device="cuda")

    def go():
        api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s, bias=c.bias, act="silu", residual=c.res, save="z8", z=z8,
                                 out=y, workspace=wf)
        api.act8_quantize(c.x, out=x8)
        api.qlora_linear_act_bwd(c.dy, c.qw, c.a, c.b, c.s, act="silu", x=x8, z=z8, lora_grads=True, bias_grad=True,
                                 dx=dx, d_lora_a=da, d_lora_b=db, d_bias=dbias, workspace=wb)
    outs = [y, dx, da, db, dbias]
    go()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        go()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for k in range(4):
        c.x.copy_(torch.randn_like(c.x, dtype=torch.float32))
        go()
        torch.cuda.synchronize()
        ref = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, outs):
            assert torch.equal(a, b), k


@pytest.mark.parametrize("T,N,K", [(2048, 22016, 64), (2000, 21952, 128), (2048, 11008, 64), (1000, 11008, 64),
                                   (700, 16384, 64), (130, 320, 128)])
def test_tile_mixes(T, N, K):
    """Grids whose last round takes smaller token tiles: two full rounds then 192 (22016 columns at
    2048 tokens, and ragged in both directions), one then 128, a round without a mix, and single
    rounds of 192 and 128 tokens.  Forward with an epilogue and without, and dX of the transposed shape with and
    without a gradient to add."""
    say(f"[tile mix] T={T} N={N} K={K}")
    c = Case(T, N, K, 8)
    y = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s, bias=c.bias, act="silu", mul=c.mul, residual=c.res)
    p = api.qlora_linear_fwd(c.x, c.qw, c.a, c.b, c.s)
    torch.cuda.synchronize()
    check(y, oracle.act_fwd(f64(c.x), c.wd, *c.ab64(), c.s, f64(c.bias), "silu", f64(c.mul), f64(c.res))[0], "Y")
    check(p, oracle.act_fwd(f64(c.x), c.wd, *c.ab64(), c.s)[0], "plain Y")
    d = Case(T, K, N, 8)                                     # K outputs, N inputs: dX is [T, N]
    g = api.qlora_linear_act_bwd(d.dy, d.qw, d.a, d.b, d.s, dx_add=d.add)
    dx = api.qlora_linear_bwd_input(d.dy, d.qw, d.a, d.b, d.s)[0]
    torch.cuda.synchronize()
    ref = oracle.act_bwd(f64(d.dy), d.wd, *d.ab64(), d.s)
    check(dx, ref["dx"], "plain dX")
    check(g.dx, ref["dx"] + f64(d.add), "dX")
