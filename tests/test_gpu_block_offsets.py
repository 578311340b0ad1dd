"""The norm, the 8-bit rows and the 8-bit product on tensors whose offsets pass 32 bits (in
elements of the norm's and the rows' 16-bit values, in bytes of a weight's codes).

The inputs repeat one block of rows, so every block of the outputs has to repeat the first,
which is compared with the same call on one block alone: bit for bit, since a row's result
depends on nothing else.  About 35 GB of GPU memory."""
import pytest
import torch

from qlora_linear_layers_amd import api
from helpers import say

pytestmark = pytest.mark.gpu

D, BLOCK, TIMES = 4096, 2100, 500            # 4.3e9 values


def block(seed, dt=torch.bfloat16, cols=D):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((BLOCK, cols), generator=g, device="cuda").to(dt)


def repeats(big, one):
    """Every block of `big` has the bits of `one`."""
    one = one.contiguous().view(torch.int16)
    parts = big.view(torch.int16).view(TIMES, *one.shape)
    return all(torch.equal(p, one) for p in parts)


def test_norm_past_32_bits():
    say(f"[offsets] norm of {BLOCK * TIMES} x {D}")
    x1, r1, w = block(1), block(2), torch.randn(D, device="cuda")
    x, r = x1.repeat(TIMES, 1), r1.repeat(TIMES, 1)
    assert x.numel() > 1 << 32
    y1, h1 = api.rmsnorm_fwd(x1, w, residual=r1)
    y, h = api.rmsnorm_fwd(x, w, residual=r, h=r)          # in place of the residual
    assert repeats(y, y1) and repeats(h, h1)
    del y, r, h
    g1 = api.rmsnorm_bwd(x1, h1, w, dx_add=x1, weight_grad=False)
    h = h1.repeat(TIMES, 1)
    g = api.rmsnorm_bwd(x, h, w, dx_add=x, dx=x)
    assert repeats(g.dx, g1.dx)
    # dw is TIMES that of one block: at most 4200 additions in a team, 30 between them
    n = h1.double() * (h1.double().square().mean(1, keepdim=True) + 1e-6).rsqrt()
    terms = x1.double() * n
    bound = 2.0 ** -24 * 4300 * terms.abs().sum(0) * TIMES
    assert bool(((g.d_weight.double() - terms.sum(0) * TIMES).abs() <= bound).all())


def test_rows_past_32_bits():
    say(f"[offsets] rows of {BLOCK * TIMES} x {D}")
    x1 = block(3, torch.float16)
    x1[:, ::50] *= 20
    q1 = api.rows8_quantize(x1)
    q = api.rows8_quantize(x1.repeat(TIMES, 1))
    assert q.codes.numel() > 1 << 32
    assert repeats(q.codes, q1.codes) and torch.equal(q.scale, q1.scale.repeat(TIMES))
    back = api.rows8_dequantize(q, dtype=torch.float16)
    assert repeats(back, api.rows8_dequantize(q1, dtype=torch.float16))


@pytest.mark.parametrize("T", [3, 40, 300])
def test_weight_past_32_bits(T):
    """A weight of 2^20 channels whose codes take more than 2^32 bytes, on the decode kernel and on tiles."""
    say(f"[offsets] product of {T} tokens with 2^20 channels")
    N, K = 1 << 20, 4200
    w1 = api.rows8_quantize(block(4, cols=K))
    codes = w1.codes.repeat(-(-N // BLOCK), 1)[:N]
    scale = w1.scale.repeat(-(-N // BLOCK))[:N]
    assert codes.numel() > 1 << 32
    x8 = api.rows8_quantize(block(5, cols=K)[:T].clone())
    y1 = api.int8_linear_fwd(x8, w1)
    y = api.int8_linear_fwd(x8, api.Rows8(codes, scale, (N, K)))
    for n in range(0, N, BLOCK):
        assert torch.equal(y[:, n:n + BLOCK], y1[:, :min(BLOCK, N - n)]), n
