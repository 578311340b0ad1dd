"""The norm and its backward at the ends of fp32: mean squares and eps below the normal
range, and gradients whose products with h leave it.

The bounds are those of test_gpu_block.py: they count the roundings of fp32 steps whose
values stay in its normal range, which is what the kernels' scaling is for.  A rest of
2^-149 per step where a result itself is that small is inside TINY (half the step of the
type's subnormals, 2^-134 for bf16 and 2^-25 for fp16)."""
import numpy as np
import pytest
import torch

import oracle
from qlora_linear_layers_amd import api
from helpers import say
from test_gpu_block import DT, TINY, U, bwd_bound, f64, make, norm_bound, within

pytestmark = pytest.mark.gpu

SIZES = [8, 64, 1000, 5000, 8192, 9000, 16391, 20000]      # every team of both kernels
EPS = [2.0 ** -149, 1e-40, 2.0 ** -126, 1e-30, 1e-12]


def small_rows(D, dt, seed):
    """Zeros, the type's smallest value, rows of shrinking size, one of ordinary size, and one whose values span it all."""
    x = make(seed)(8, D, dt=torch.float32)
    x[0] = 0
    x[1] = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    for i, s in ((2, 1e-38), (3, 1e-25), (4, 3e-20), (5, 1e-15)):
        x[i] *= s
    x[7] *= torch.logspace(-38, 0, D, device="cuda")
    return x.to(dt)


@pytest.mark.parametrize("D", SIZES)
@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_tiny_mean_squares(D, eps, dtype):
    """An eps and rows whose squares lie below fp32's normal range: a row of zeros gives zeros, and the
    rest what the formula gives, in both directions."""
    say(f"[norm range] D={D} eps={eps} {dtype}")
    dt, e32 = DT[dtype], float(np.float32(eps))
    x, w = small_rows(D, dt, D), (1 + 0.3 * make(D + 1)(D, dt=torch.float32))
    y = api.rmsnorm_fwd(x, w, eps)
    y8 = api.rmsnorm_fwd(x, w, eps, quantize=True)
    torch.cuda.synchronize()
    ref = oracle.rmsnorm(f64(x), f64(w), eps)
    within(y, ref, norm_bound(ref, dt), "y")
    assert not f64(y)[0].any()
    d = f64(y8.scale)[:, None]
    rd = np.abs(ref).max(1, keepdims=True) / 127
    zero = rd * 127 < 2.0 ** -120 * (1 + 1e-5)             # stored as zeros below 2^-120
    within(d, rd, np.where(zero, rd, 5e-6 * rd), "scale")
    within(f64(y8.codes)[:, :D] * d, ref, np.where(zero, np.abs(ref), rd * (0.5 + 2e-3)), "codes")

    dy = make(D + 2)(8, D, dt=dt)
    scale = 1.0
    if dt == torch.float16:
        # fp16 holds gradients up to 65504: dY is small where the norm's slope is large
        scale = min(1.0, 1e3 * eps ** 0.5)
        dy = torch.zeros_like(dy) if scale < 2.0 ** -24 else (dy.float() * scale).to(dt)
    g = api.rmsnorm_bwd(dy, x, w, eps)
    torch.cuda.synchronize()
    rdx, rdw = oracle.rmsnorm_bwd(f64(dy), f64(x), f64(w), eps)
    within(g.dx, rdx, bwd_bound(rdx, f64(dy), f64(x), f64(w), e32, dt), "dx")
    terms = np.abs(f64(dy) * oracle.rmsnorm(f64(x), None, eps)).sum(0)
    within(g.d_weight, rdw, U[torch.float32] * np.abs(rdw) + 1e-5 * terms + TINY[torch.float32], "dw")


@pytest.mark.parametrize("D", [1, 2, 70, 5000])
def test_eps_as_large_as_the_squares(D):
    """The sum of eps and the squares leaves fp32 where neither does."""
    say(f"[norm range] large eps D={D}")
    dt, eps = torch.bfloat16, 3e38
    x = torch.full((3, D), 1.2e19 / D ** 0.5, device="cuda")
    x[1] *= -0.5
    x[2] = 1.0
    x, dy, w = x.to(dt), make(D)(3, D, dt=dt) * 2.0 ** 40, make(D + 1)(D, dt=torch.float32)
    y = api.rmsnorm_fwd(x, w, eps)
    g = api.rmsnorm_bwd(dy, x, w, eps)
    torch.cuda.synchronize()
    ref = oracle.rmsnorm(f64(x), f64(w), eps)
    within(y, ref, norm_bound(ref, dt), "y")
    rdx, rdw = oracle.rmsnorm_bwd(f64(dy), f64(x), f64(w), eps)
    within(g.dx, rdx, bwd_bound(rdx, f64(dy), f64(x), f64(w), float(np.float32(eps)), dt), "dx")
    terms = np.abs(f64(dy) * oracle.rmsnorm(f64(x), None, eps)).sum(0)
    within(g.d_weight, rdw, U[torch.float32] * np.abs(rdw) + 1e-5 * terms + TINY[torch.float32], "dw")


@pytest.mark.parametrize("D", SIZES)
@pytest.mark.parametrize("h_size,dy_size", [(2.0 ** 33, 2.0 ** 100), (2.0 ** 100, 2.0 ** 100), (1.0, 2.0 ** 120),
                                            (2.0 ** 120, 2.0 ** 90)])
@pytest.mark.parametrize("weight", [True, False])
def test_gradients_whose_products_leave_fp32(D, h_size, dy_size, weight):
    """dY h beyond 2^128 where dx and dw are ordinary numbers: mean(g n) is formed from n."""
    say(f"[norm range] D={D} h about {h_size:g} dy about {dy_size:g} weight={weight}")
    dt, n, T = torch.bfloat16, make(D), 5
    h, dy = n(T, D, dt=torch.float32), n(T, D, dt=torch.float32)
    h[1:4] *= h_size                                       # an ordinary row before and behind them
    dy[1:4] *= dy_size
    h, dy = h.to(dt), dy.to(dt)
    w = (1 + 0.3 * n(D, dt=torch.float32)) if weight else None
    g = api.rmsnorm_bwd(dy, h, w, 1e-6)
    torch.cuda.synchronize()
    e32, wv = float(np.float32(1e-6)), None if w is None else f64(w)
    rdx, rdw = oracle.rmsnorm_bwd(f64(dy), f64(h), wv, 1e-6)
    within(g.dx, rdx, bwd_bound(rdx, f64(dy), f64(h), wv, e32, dt), "dx")
    if w is not None:
        terms = np.abs(f64(dy) * oracle.rmsnorm(f64(h), None, 1e-6)).sum(0)
        within(g.d_weight, rdw, U[torch.float32] * np.abs(rdw) + 1e-5 * terms + TINY[torch.float32], "dw")
