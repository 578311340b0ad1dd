"""The norm, the 8-bit rows and the 8-bit product on the GPU, against the fp64 oracle.

Tolerances, u the half step of a 16-bit type (2^-8 bf16, 2^-11 fp16) and tiny half
the step of its subnormals (fp16 2^-25, bf16 2^-134):
  rows8      codes, scales and values bit for bit.
  norm       h bit for bit.  y: the sum of squares has at most 8 x 8 + 16 additions in
             sequence, 80 roundings of 2^-24, half of them through the root; the root,
             the division and three products add five.  45 x 2^-24 < 4e-6 relative, and
             one rounding: |y - ref| <= (u + 4e-6) |ref| + tiny.  In 8 bits: a code is off
             by half a unit, by 127 x 4e-6 twice over (value and unit), 127 x 2^-22 for
             the factor: d (0.5 + 2e-3); the unit itself by 5e-6.
  backward   dx: mean(g n) is a sum of the same kind, off by 6e-6 mean|g n|; then a few
             roundings of the terms: u |dx| + 1e-5 r (|g| + |n| mean|g n|) + 2^-23 |add|.
             dw: at most T / teams + teams / 16 + 16 additions in sequence, below 110 for the
             sizes here: u |dw| (none in fp32) + 1e-5 sum|dy n|.
  product    without an epilogue the value is fl32(fl32(fl32(sum) min) max) rounded once:
             bit for bit.  With one: the fp32 steps (at most ten roundings, the activation's
             1e-5 relative at most) on z, bias, act, mul and res:
             u |y| + 2e-5 (|z| + |bias| + |act|) |mul| + 2^-23 |res| + tiny."""
import numpy as np
import pytest
import torch

import oracle
from qlora_linear_layers_amd import api
from helpers import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def f64(t):
    return t.detach().double().cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def round16(v, dt):
    """Bits of fp64 values rounded once to a 16-bit type."""
    return oracle.round_to_f16_bits(v) if dt == torch.float16 else oracle.round_to_bf16_bits(v)


def within(got, ref, bound, what):
    g, ref = f64(got) if isinstance(got, torch.Tensor) else got, np.asarray(ref)
    assert g.shape == ref.shape, what
    assert np.isfinite(g).all(), what
    over = np.abs(g - ref) - bound
    say(f"  {what}: worst {float(np.max(np.abs(g - ref) / np.maximum(bound, 1e-300))):.3f} of the bound")
    assert float(over.max()) <= 0, what


def make(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *sh, std=1.0, dt=torch.bfloat16: (torch.randn(sh, generator=g) * std).to(dt).cuda()


def behind(rows, cols, dt, extra=3):
    """(a tensor [rows, cols], a check that what lies behind it is as it was)."""
    big = torch.full(((rows + extra) * cols,), 77.0, device="cuda").to(dt)
    return big[:rows * cols].view(rows, cols), lambda: bool((big[rows * cols:] == 77).all())


# ------------------------------------------------------------------ rows in 8 bits

# every team (one wave, 256 and 1024 threads) and chunk count, odd lengths, a last group of rows part empty
ROWS = [(1, 1), (3, 7), (5, 64), (6, 129), (9, 512), (3, 513), (7, 1000), (5, 1531), (2, 2048), (3, 2049), (2, 4099),
        (3, 8192), (2, 11008), (3, 16385), (2, 22016), (1, 32769), (2, 65536), (1027, 96)]


@pytest.mark.parametrize("R,K", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rows8(R, K, dtype):
    say(f"[rows8] {R} x {K} {dtype}")
    dt = DT[dtype]
    x = make(R + K)(R, K, dt=dt)
    x[:, ::37] *= 20
    codes, codes_ok = behind(R, api.rows8_pitch(K), torch.int8)
    scale, scale_ok = behind(R, 1, torch.float32)
    back, back_ok = behind(R, K, dt)
    r8 = api.rows8_quantize(x, out=api.Rows8(codes, scale.view(R), (R, K)))
    api.rows8_dequantize(r8, out=back)
    torch.cuda.synchronize()
    rq, rd = oracle.rows8_quantize(f64(x))
    assert np.array_equal(codes.cpu().numpy(), rq)
    assert np.array_equal(scale.cpu().numpy().reshape(-1).view(np.uint32), rd.view(np.uint32))
    assert np.array_equal(bits(back).reshape(R, K), round16(oracle.rows8_values(rq, rd, K), dt).reshape(R, K))
    assert codes_ok() and scale_ok() and back_ok()
    assert r8.nbytes() == R * (api.rows8_pitch(K) + 4)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K", [70, 3000, 20000])
def test_rows8_special_rows(K, dtype):
    say(f"[rows8] special rows K={K} {dtype}")
    dt = DT[dtype]
    x = torch.ones((8, K), dtype=dt)
    x[0] = 0
    x[1, K - 1] = float("inf")
    x[2, 3] = float("nan")
    x[3, 0] = float("-inf")
    x[4] = torch.finfo(dt).max
    x[5] = torch.finfo(dt).smallest_normal            # bf16: below 2^-120, zeros
    x[6] = torch.arange(K) % 255 - 127.0              # exact codes, and ties with the next row's unit
    x[7] = (torch.arange(K) % 255 - 127.0) * 0.5
    x[7, 5] = 127.0
    r8 = api.rows8_quantize(x.cuda())
    torch.cuda.synchronize()
    rq, rd = oracle.rows8_quantize(x.double().numpy())
    assert np.array_equal(r8.codes.cpu().numpy(), rq)
    d = r8.scale.cpu().numpy()
    assert np.array_equal(np.isnan(d), np.isnan(rd)) and np.isnan(d[1:4]).all()
    assert np.array_equal(np.delete(d, [1, 2, 3]), np.delete(rd, [1, 2, 3]))
    back = f64(api.rows8_dequantize(r8, dtype=dt))
    assert np.isnan(back[1:4]).all() and np.isfinite(np.delete(back, [1, 2, 3], 0)).all()


# ------------------------------------------------------------------ the norm

NORMS = [(1, 1), (2, 8), (5, 100), (3, 512), (9, 777), (6, 1024), (5, 2047), (3, 2050), (1, 4096), (3, 4099), (2, 8192),
         (2, 8200), (3, 16391), (1, 32768), (1030, 64)]


def norm_bound(ref, dt):
    return (U[dt] + 4e-6) * np.abs(ref) + TINY[dt]


@pytest.mark.parametrize("T,D", NORMS)
@pytest.mark.parametrize("dtype,residual,weight", [("bf16", True, "16"), ("bf16", False, "32"), ("fp16", True, "32"),
                                                   ("fp16", False, None), ("bf16", True, None)])
def test_norm(T, D, dtype, residual, weight):
    say(f"[norm] {T} x {D} {dtype} residual={residual} weight={weight}")
    dt, n = DT[dtype], make(T + D)
    x, res = n(T, D, dt=dt), n(T, D, dt=dt) if residual else None
    x[:, ::41] *= 15
    w = None if weight is None else (1 + 0.3 * n(D, dt=torch.float32)).to(dt if weight == "16" else torch.float32)
    eps = 1e-5
    y, y_ok = behind(T, D, dt)
    h, h_ok = behind(T, D, dt)
    got = api.rmsnorm_fwd(x, w, eps, residual=res, h=h if residual else None, out=y)
    y8 = api.rmsnorm_fwd(x, w, eps, residual=res, quantize=True, keep_h=False)
    torch.cuda.synchronize()
    assert (got[0] is y and got[1] is h) if residual else got is y
    assert y_ok() and h_ok()
    if residual:
        assert np.array_equal(bits(h).reshape(T, D), round16(f64(x) + f64(res), dt).reshape(T, D))
    hv = f64(h) if residual else f64(x)
    ref = oracle.rmsnorm(hv, None if w is None else f64(w), eps)
    within(y, ref, norm_bound(ref, dt), "y")
    # 8 bits of the unrounded y
    d = f64(y8.scale)[:, None]
    rd = np.abs(ref).max(1, keepdims=True) / 127
    within(d, rd, 5e-6 * rd, "scale")
    q = f64(y8.codes)
    assert not q[:, D:].any() and (np.abs(q).max(1) == 127).all()
    within(q[:, :D] * d, ref, rd * (0.5 + 2e-3), "codes")


@pytest.mark.parametrize("D", [96, 4100, 9001])
def test_norm_writes_both_and_in_place(D):
    """The C entry writes 16 and 8 bits at once; h may be x or the residual."""
    say(f"[norm] both outputs, in place, D={D}")
    T, n = 37, make(D)
    x, res, w = n(T, D), n(T, D), n(D)
    y, h = api.rmsnorm_fwd(x, w, residual=res)
    y8, h8 = api.rmsnorm_fwd(x, w, residual=res, quantize=True)
    both, b8 = torch.empty_like(x), api.rows8_empty((T, D))
    assert api.lib().rmsnorm_fwd(x.data_ptr(), res.data_ptr(), T, D, w.data_ptr(), 0, 1e-6, None, both.data_ptr(),
                                 b8.codes.data_ptr(), b8.scale.data_ptr(), api._stream()) == 0
    for where in ("x", "res"):
        t = {"x": x.clone(), "res": res.clone()}
        y2, h2 = api.rmsnorm_fwd(t["x"], w, residual=t["res"], h=t[where])
        assert h2 is t[where] and torch.equal(y2, y) and torch.equal(h2, h), where
    torch.cuda.synchronize()
    assert torch.equal(both, y) and torch.equal(b8.codes, y8.codes) and torch.equal(b8.scale, y8.scale)
    assert torch.equal(h8, h)


@pytest.mark.parametrize("D", [64, 5000])
def test_norm_over_the_types_range(D):
    """Rows of zeros, of huge values (whose squares leave fp32), of the smallest, and rows with an inf
    or a NaN: inf gives NaN there and 0 beside it, a NaN the whole row; in 8 bits both read NaN."""
    say(f"[norm] range D={D}")
    dt, w = torch.bfloat16, torch.full((D,), 0.5, dtype=torch.bfloat16, device="cuda")
    x = make(D)(8, D)
    x[1] = 0
    x[2] *= 1e30
    x[3] = torch.finfo(dt).max
    x[4] *= 1e-30
    x[5, 7] = float("inf")
    x[6, 9] = float("nan")
    x[7] *= 2.0 ** 64
    y = api.rmsnorm_fwd(x, w)
    y8 = api.rows8_dequantize(api.rmsnorm_fwd(x, w, quantize=True))
    dy = make(D + 1)(8, D)
    g = api.rmsnorm_bwd(dy, x, w)
    torch.cuda.synchronize()
    fine = [0, 1, 2, 3, 4, 7]
    ref = oracle.rmsnorm(f64(x)[fine], f64(w), 1e-6)
    within(f64(y)[fine], ref, norm_bound(ref, dt), "y")
    assert np.isfinite(f64(y8)[fine]).all()
    yn = f64(y)
    assert np.isnan(yn[5, 7]) and (np.delete(yn[5], 7) == 0).all() and np.isnan(yn[6]).all()
    assert np.isnan(f64(y8)[5:7]).all()
    # an eps as large as such rows' mean square counts there, too
    e = api.rmsnorm_fwd(x[7:8].contiguous(), w, 3e38)
    ref = oracle.rmsnorm(f64(x)[7:8], f64(w), 3e38)
    within(e, ref, norm_bound(ref, dt), "y with a large eps")
    hv, dv = f64(x)[fine], f64(dy)[fine]
    rdx = oracle.rmsnorm_bwd(dv, hv, f64(w), 1e-6)[0]
    within(f64(g.dx)[fine], rdx, bwd_bound(rdx, dv, hv, f64(w), 1e-6, dt), "dx")


def bwd_bound(ref, dy, h, w, eps, dt, add=None):
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    n, gr = h * r, np.abs(dy if w is None else dy * w)
    b = U[dt] * np.abs(ref) + 1e-5 * r * (gr + np.abs(n) * (gr * np.abs(n)).mean(1, keepdims=True)) + TINY[dt]
    return b if add is None else b + 2.0 ** -23 * np.abs(add)


@pytest.mark.parametrize("T,D", NORMS + [(300, 8192), (1500, 1024), (777, 3001)])
@pytest.mark.parametrize("dtype,add,weight", [("bf16", True, "16"), ("fp16", False, "32"), ("bf16", False, None),
                                              ("fp16", True, "16")])
def test_norm_backward(T, D, dtype, add, weight):
    say(f"[norm bwd] {T} x {D} {dtype} add={add} weight={weight}")
    dt, n = DT[dtype], make(T + D)
    h, dy, ad = n(T, D, dt=dt), n(T, D, dt=dt), n(T, D, dt=dt) if add else None
    h[:, ::41] *= 15
    w = None if weight is None else (1 + 0.3 * n(D, dt=torch.float32)).to(dt if weight == "16" else torch.float32)
    dx, dx_ok = behind(T, D, dt)
    g = api.rmsnorm_bwd(dy, h, w, 1e-5, dx_add=ad, dx=dx)
    g2 = api.rmsnorm_bwd(dy, h, w, 1e-5, dx_add=ad, weight_grad=False)
    torch.cuda.synchronize()
    assert dx_ok() and g2.d_weight is None and torch.equal(g2.dx, g.dx)
    wv, av = None if w is None else f64(w), None if ad is None else f64(ad)
    rdx, rdw = oracle.rmsnorm_bwd(f64(dy), f64(h), wv, 1e-5, av)
    within(g.dx, rdx, bwd_bound(rdx, f64(dy), f64(h), wv, 1e-5, dt, av), "dx")
    if w is None:
        assert g.d_weight is None
        return
    assert g.d_weight.dtype == w.dtype
    terms = np.abs(f64(dy) * oracle.rmsnorm(f64(h), None, 1e-5)).sum(0)
    within(g.d_weight, rdw, U[w.dtype] * np.abs(rdw) + 1e-5 * terms + TINY[w.dtype], "dw")
    # the same bits again, and in place of dy and of dx_add
    again = api.rmsnorm_bwd(dy, h, w, 1e-5, dx_add=ad, dx=dy.clone())
    assert torch.equal(again.dx, g.dx) and torch.equal(again.d_weight, g.d_weight)
    t = dy.clone()
    assert torch.equal(api.rmsnorm_bwd(t, h, w, 1e-5, dx_add=ad, dx=t).dx, g.dx)
    if add:
        t = ad.clone()
        assert torch.equal(api.rmsnorm_bwd(dy, h, w, 1e-5, dx_add=t, dx=t).dx, g.dx)


# Sizes whose rows pass by the caches (2^24 values in the forward, 2^25 in the backward): rows
# of one call do not depend on each other, so a few of them alone give the same bits.
@pytest.mark.parametrize("T,D,dtype", [(2049, 8192, "bf16"), (2050, 8193, "fp16"), (16397, 1024, "bf16"),
                                       (1025, 16392, "bf16")])
@pytest.mark.parametrize("quantize", [False, True])
def test_norm_of_large_batches(T, D, dtype, quantize):
    say(f"[norm, large] {T} x {D} {dtype} quantize={quantize}")
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(T + D)
    x, res = (torch.randn((T, D), generator=g, device="cuda").to(dt) for _ in range(2))
    w = torch.randn(D, generator=g, device="cuda").to(dt)
    h, h_kept = behind(T, D, dt)
    y, _ = api.rmsnorm_fwd(x, w, 1e-5, residual=res, quantize=quantize, h=h)
    for lo, hi in ((0, 9), (T // 2, T // 2 + 5), (T - 7, T)):
        ys, hs = api.rmsnorm_fwd(x[lo:hi].clone(), w, 1e-5, residual=res[lo:hi].clone(), quantize=quantize)
        assert torch.equal(h[lo:hi].view(torch.int16), hs.view(torch.int16))
        if quantize:
            assert torch.equal(y.codes[lo:hi], ys.codes) and torch.equal(y.scale[lo:hi], ys.scale)
        else:
            assert torch.equal(y[lo:hi].view(torch.int16), ys.view(torch.int16))
    assert torch.equal(h.view(torch.int16), (x.float() + res.float()).to(dt).view(torch.int16))
    assert h_kept()


@pytest.mark.parametrize("T,D,dtype", [(4099, 8192, "bf16"), (8197, 4104, "fp16"), (32771, 1024, "bf16"),
                                       (4099, 8193, "bf16"), (2050, 16384, "bf16")])
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_backward_of_large_batches(T, D, dtype, in_place):
    say(f"[norm backward, large] {T} x {D} {dtype} in_place={in_place}")
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(T + D)
    dy, h, add = (torch.randn((T, D), generator=g, device="cuda").to(dt) for _ in range(3))
    w = torch.randn(D, generator=g, device="cuda")
    dy0 = dy.clone()
    got = api.rmsnorm_bwd(dy, h, w, 1e-5, dx_add=add, dx=dy if in_place else None)
    for lo, hi in ((0, 9), (T // 2, T // 2 + 5), (T - 7, T)):
        few = api.rmsnorm_bwd(dy0[lo:hi].clone(), h[lo:hi].clone(), w, 1e-5, dx_add=add[lo:hi].clone())
        assert torch.equal(got.dx[lo:hi].view(torch.int16), few.dx.view(torch.int16))
    ref, size = (torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(2))
    for lo in range(0, T, 1024):
        hd = h[lo:lo + 1024].double()
        n = dy0[lo:lo + 1024].double() * hd * (hd.square().mean(1, keepdim=True) + 1e-5).rsqrt()
        ref += n.sum(0)
        size += n.abs().sum(0)
    within(got.d_weight, f64(ref), U[torch.float32] * np.abs(f64(ref)) + 1e-5 * f64(size), "dw")


def test_norm_gradient_against_differences():
    """The kernel's dx and dw against differences of the definition along random directions."""
    say("[norm bwd] differences")
    T, D, dt, n = 6, 200, torch.float16, make(3)
    h, dy, w = n(T, D, dt=dt), n(T, D, dt=dt), n(D, dt=torch.float32)
    g = api.rmsnorm_bwd(dy, h, w, 1e-5)
    torch.cuda.synchronize()
    rng, step = np.random.default_rng(0), 1e-5
    loss = lambda hv, wv: float((oracle.rmsnorm(hv, wv, 1e-5) * f64(dy)).sum())
    for _ in range(4):
        eh, ew = rng.standard_normal((T, D)), rng.standard_normal(D)
        for got, e, f in ((g.dx, eh, lambda s: loss(f64(h) + s * eh, f64(w))),
                          (g.d_weight, ew, lambda s: loss(f64(h), f64(w) + s * ew))):
            diff = (f(step) - f(-step)) / (2 * step)
            gv = f64(got)
            # each element off by its rounding; the difference quotient by about step^2
            assert abs(float((gv * e).sum()) - diff) <= float((np.abs(gv * e)).sum()) * 2.0 ** -11 + 1e-5


# ------------------------------------------------------------------ the 8-bit product

def rows8_of(n, R, K, std=1.0):
    x = n(R, K, std=std, dt=torch.float32)
    codes, d = oracle.rows8_quantize(f64(x))
    return api.Rows8(torch.from_numpy(codes).cuda(), torch.from_numpy(d).cuda(), (R, K))


def product_bits(x8, w8, dt):
    """Bits of fl32(fl32(fl32(sum) min) max) rounded once."""
    s = (x8.codes.cpu().numpy().astype(np.float64) @ w8.codes.cpu().numpy().astype(np.float64).T).astype(np.float32)
    a, b = x8.scale.cpu().numpy()[:, None], w8.scale.cpu().numpy()[None, :]
    return round16(((s * np.minimum(a, b)) * np.maximum(a, b)).astype(np.float64), dt).reshape(s.shape)


# token counts around the decode kernel's groups and the edges of 64- and 128-token tiles (products of more tiles:
# test_gpu_block_routes.py); channels and lengths from one on, odd ones among them
PRODUCTS = [(1, 1, 1), (1, 70, 5), (2, 64, 128), (3, 17, 64), (15, 100, 127), (16, 256, 129), (17, 33, 300), (32, 320, 256),
            (33, 130, 1000), (48, 1000, 512), (64, 64, 640), (65, 257, 384), (100, 512, 1024), (129, 300, 4099),
            (200, 1024, 2048), (256, 256, 256), (257, 511, 130), (300, 4097, 777), (513, 200, 1280), (777, 1024, 512),
            (5, 4096, 11008), (1030, 1100, 320), (40, 128, 20000), (2100, 9, 33)]


@pytest.mark.parametrize("T,N,K", PRODUCTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_product_bits(T, N, K, dtype):
    say(f"[int8] T={T} N={N} K={K} {dtype}")
    n, dt = make(T + N + K), DT[dtype]
    x8, w8 = rows8_of(n, T, K), rows8_of(n, N, K, std=K ** -0.5)
    y, y_ok = behind(T, N, dt)
    api.int8_linear_fwd(x8, w8, out=y)
    torch.cuda.synchronize()
    assert np.array_equal(bits(y).reshape(T, N), product_bits(x8, w8, dt))
    assert y_ok()


@pytest.mark.parametrize("T,N,K", [(1, 70, 65), (7, 256, 512), (20, 129, 300), (64, 320, 128), (130, 264, 384),
                                   (300, 513, 640), (600, 1024, 256), (1025, 384, 1000)])
@pytest.mark.parametrize("act", oracle.ACTS)
@pytest.mark.parametrize("dtype,bias,mul,res", [("bf16", False, True, False), ("fp16", True, False, True),
                                                ("bf16", True, True, True)])
def test_product_epilogue(T, N, K, act, dtype, bias, mul, res):
    say(f"[int8] epilogue T={T} N={N} K={K} {act} {dtype} bias={bias} mul={mul} res={res}")
    n, dt = make(T + N + K), DT[dtype]
    x8, w8 = rows8_of(n, T, K), rows8_of(n, N, K, std=2 * K ** -0.5)
    b, m, r = (n(N, dt=dt) if bias else None, n(T, N, dt=dt) if mul else None, n(T, N, dt=dt) if res else None)
    y, y_ok = behind(T, N, dt)
    api.int8_linear_fwd(x8, w8, bias=b, act=act, mul=m, residual=r, out=y)
    torch.cuda.synchronize()
    assert y_ok()
    o = lambda t: None if t is None else f64(t)
    ry, rz = oracle.int8_linear(x8.codes.cpu().numpy(), f64(x8.scale), w8.codes.cpu().numpy(), f64(w8.scale), o(b), act,
                                o(m), o(r))
    mag = np.abs(rz) + np.abs(oracle.act(rz, act)) + (0 if b is None else np.abs(o(b)))
    bound = U[dt] * np.abs(ry) + 2e-5 * mag * (1 if m is None else np.abs(o(m))) + TINY[dt]
    within(y, ry, bound + (0 if r is None else 2.0 ** -23 * np.abs(o(r))), "y")
    for where in ("mul", "residual"):                  # y in the buffer of either
        t = {"mul": m, "residual": r}
        if t[where] is None:
            continue
        t = {k: None if v is None else v.clone() for k, v in t.items()}
        assert torch.equal(api.int8_linear_fwd(x8, w8, bias=b, act=act, out=t[where], **t), y), where


@pytest.mark.parametrize("T,N,K", [(2, 40, 65536), (20, 33, 65536), (300, 300, 65536)])
def test_product_of_extreme_codes(T, N, K):
    """The longest rows of the largest codes: the sum comes near 2^30 and stays exact."""
    say(f"[int8] extreme codes T={T} N={N} K={K}")
    x8 = api.Rows8(torch.full((T, K), 127, dtype=torch.int8, device="cuda"), torch.ones(T, device="cuda"), (T, K))
    w8 = api.Rows8(torch.full((N, K), -127, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"), (N, K))
    x8.codes[1] = -127
    w8.codes[::2, ::3] = 126
    y = api.int8_linear_fwd(x8, w8)
    torch.cuda.synchronize()
    assert np.array_equal(bits(y).reshape(T, N), product_bits(x8, w8, torch.bfloat16))


@pytest.mark.parametrize("T", [3, 40, 200])
def test_product_scales(T):
    """Rows of zeros, NaN scales (a whole row, a whole column), scales at the ends of fp32."""
    say(f"[int8] scales T={T}")
    n, N, K = make(T), 90, 200
    x8, w8 = rows8_of(n, T, K), rows8_of(n, N, K)
    x8.scale[0] = float("nan")
    w8.scale[5] = float("nan")
    x8.codes[1] = 0
    x8.scale[1] = 3e38
    w8.scale[6] = 3e38                                 # 0 times an overflowing product of scales is 0
    x8.scale[2] = 1e-38
    w8.scale[7] = 1e30                                 # a tiny scale times a large one
    y = f64(api.int8_linear_fwd(x8, w8))
    torch.cuda.synchronize()
    assert np.isnan(y[0]).all() and np.isnan(y[:, 5]).all()
    assert (np.delete(y[1], 5) == 0).all()
    s = x8.codes[2].double() @ w8.codes[7].double()
    ref = float(s) * float(x8.scale[2].double() * w8.scale[7].double())
    assert abs(y[2, 7] - ref) <= 2.0 ** -8 * abs(ref) * 1.001
    assert not np.isnan(np.delete(np.delete(y, 0, 0), 5, 1)).any()


# ------------------------------------------------------------------ together, on streams, in graphs

def block_calls(x, res, w, up, down, out):
    """The operators in a row, as a block calls them: norm to 8 bits, product, rows, product + residual."""
    x8, h = api.rmsnorm_fwd(x, w, residual=res, quantize=True)
    u = api.int8_linear_fwd(x8, up, act="silu")
    return api.int8_linear_fwd(api.rows8_quantize(u), down, residual=h, out=out)


@pytest.mark.parametrize("T,D,F", [(1, 256, 700), (33, 320, 513), (300, 512, 1024)])
def test_a_run_of_them_on_another_stream_and_in_a_graph(T, D, F):
    say(f"[block] T={T} D={D} F={F}")
    n = make(T + D)
    x, res, w = n(T, D), n(T, D), n(D)
    up, down = api.rows8_quantize(n(F, D, std=D ** -0.5)), api.rows8_quantize(n(D, F, std=F ** -0.5))
    ref = block_calls(x, res, w, up, down, None)
    torch.cuda.synchronize()
    # the same values from the parts' definitions: 8-bit inputs as the kernels left them
    x8, h = api.rmsnorm_fwd(x, w, residual=res, quantize=True)
    u = api.int8_linear_fwd(x8, up, act="silu")
    ru = oracle.int8_linear(x8.codes.cpu().numpy(), f64(x8.scale), up.codes.cpu().numpy(), f64(up.scale), name="silu")[0]
    within(u, ru, U[u.dtype] * np.abs(ru) + 2e-5 * (1 + np.abs(ru)) * 8, "hidden")
    side = torch.cuda.Stream()
    out = torch.zeros_like(x)
    with torch.cuda.stream(side):
        block_calls(x, res, w, up, down, out)
    side.synchronize()
    assert torch.equal(out, ref)
    # captured once, replayed on new inputs with eager work between
    with torch.cuda.stream(side):
        block_calls(x, res, w, up, down, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block_calls(x, res, w, up, down, out)
    for rep in range(3):
        x.copy_(make(rep)(T, D))
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, block_calls(x, res, w, up, down, None)), rep


def test_backward_in_a_graph():
    say("[norm bwd] graph")
    T, D, n = 700, 1024, make(5)
    dy, h, w = n(T, D), n(T, D), n(D)
    dx, dw = torch.empty_like(dy), torch.empty_like(w)
    api.rmsnorm_bwd(dy, h, w, dx=dx, d_weight=dw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.rmsnorm_bwd(dy, h, w, dx=dx, d_weight=dw)
    for rep in range(3):
        dy.copy_(make(rep)(T, D))
        dx.zero_()
        dw.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        g = api.rmsnorm_bwd(dy, h, w)
        assert torch.equal(dx, g.dx) and torch.equal(dw, g.d_weight), rep


def test_two_graphs_that_share_a_workspace():
    """Split products of two captured graphs with one workspace, replayed one after the other."""
    say("[int8] two graphs, one workspace")
    n = make(9)
    cases = [(rows8_of(n, 200, 2048), rows8_of(n, 300, 2048)), (rows8_of(n, 130, 3000), rows8_of(n, 200, 3000))]
    need = max(api.int8_linear_workspace_bytes(*a.shape, b.shape[0]) for a, b in cases)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    outs = [torch.empty((a.shape[0], b.shape[0]), dtype=torch.bfloat16, device="cuda") for a, b in cases]
    graphs = []
    for (a, b), y in zip(cases, outs):
        api.int8_linear_fwd(a, b, workspace=ws, out=y)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.int8_linear_fwd(a, b, workspace=ws, out=y)
        graphs.append(g)
    for rep in range(3):
        for y in outs:
            y.zero_()
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for (a, b), y in zip(cases, outs):
            assert torch.equal(y, api.int8_linear_fwd(a, b)), rep
