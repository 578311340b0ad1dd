"""The gated block (mlp.py) against the fp64 oracle composed the same way.

Tolerances, in the unit roundoff u of the 16-bit type (a rounding is at most
u/sqrt(3) rms).  Y: U, H and Y are rounded (three roundings, each carried on
by products that average it, and by |silu'| <= 1.1): a relative 2-norm error of
at most 3 (1.1 u/sqrt(3)) < 2 u.  The backward is held to the oracle's on the
checkpoints the forward left (read back), so only its own roundings count: dH,
dZ, dU and the sums' roundings, at most four on any path: < 2.5 u.  What the
checkpoints themselves cost is measured against the exact gradients: a code is
off by at most half a unit of max/127, about 0.7% of a block's rms for normal
values (max ~ 2.9 rms of 64: 2.9 / 127 / sqrt(12)), through X, H and the
slopes of Z and U: below 3%."""
import numpy as np
import pytest
import torch

import oracle
from qlora_linear_layers_amd import api
from qlora_linear_layers_amd.mlp import AdaptedLinear, GatedMlp
from helpers import say

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _rel(got, ref):
    return float(np.linalg.norm(_f64(got) - ref) / np.linalg.norm(ref))


def _linear(g, N, K, r, dt, s):
    n = lambda *sh, std=1.0: (torch.randn(sh, generator=g) * std).to(dt).cuda()
    qw = api.nf4_quantize_dq(n(N, K, std=1.0 / K ** 0.5))
    return AdaptedLinear(qw, n(K, r, std=0.05), n(r, N, std=0.2), s) if r else AdaptedLinear(qw)


def _w(l, dt):
    a, b = (_f64(l.lora_a), _f64(l.lora_b)) if l.lora_a is not None else (None, None)
    return _f64(api.nf4_dequantize_dq(l.qw, dtype=dt)), a, b


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,F,r,dt", [(1, 192, 320, 8, torch.bfloat16), (13, 256, 448, 16, torch.bfloat16),
                                        (50, 320, 192, 0, torch.bfloat16), (300, 256, 576, 24, torch.bfloat16),
                                        (300, 256, 576, 24, torch.float16)])
def test_block_matches_the_oracle(T, D, F, r, dt):
    say(f"[mlp] T={T} D={D} F={F} r={r} {dt}")
    g = torch.Generator().manual_seed(T + D)
    s, u = 0.5, U[dt]
    mlp = GatedMlp(_linear(g, F, D, r, dt, s), _linear(g, F, D, r, dt, s), _linear(g, D, F, r, dt, s))
    x, res, dy = ((torch.randn((T, D), generator=g)).to(dt).cuda() for _ in range(3))
    y, saved = mlp.forward_train(x, res)
    grads = mlp.backward(dy, saved)
    torch.cuda.synchronize()
    assert torch.equal(mlp.forward(x, res), y)

    wg, wu, wd = _w(mlp.gate, dt), _w(mlp.up, dt), _w(mlp.down, dt)
    ru = oracle.act_fwd(_f64(x), *wu, s)[0]
    rh, rz = oracle.act_fwd(_f64(x), *wg, s, name="silu", mul=ru)
    ry = oracle.act_fwd(rh, *wd, s, residual=_f64(res))[0]
    e = _rel(y, ry)
    say(f"  Y: {e / u:.2f} u")
    assert e < 2 * u

    def back(xv, zv, uv, hv):
        d = oracle.act_bwd(_f64(dy), *wd, s, x=hv)
        gg = oracle.act_bwd(d["dx"], *wg, s, "silu", x=xv, z=zv, mul=uv)
        uu = oracle.act_bwd(gg["dmul"], *wu, s, x=xv, dx_add=gg["dx"])
        return uu["dx"], gg, uu, d
    value = lambda a: oracle.ck_values(a.codes.cpu().numpy(), a.scale.cpu().numpy()).reshape(a.shape)
    kept = back(value(saved.x), value(saved.z), value(saved.u), value(saved.h))
    exact = back(_f64(x), rz, ru, rh)
    for what, ref, bound in (("from the checkpoints", kept, 2.5 * u), ("exact", exact, 0.03)):
        dx, gg, uu, d = ref
        pairs = [("dX", grads.dx, dx)]
        if r:
            for name, pair, o in (("gate", grads.gate, gg), ("up", grads.up, uu), ("down", grads.down, d)):
                pairs += [(name + " dA", pair[0], o["da"]), (name + " dB", pair[1], o["db"])]
        for name, got, rf in pairs:
            e = _rel(got, rf)
            say(f"  {name} against {what}: {e:.2e}")
            assert e < bound, (name, what)
    assert saved.nbytes() == sum(n + 4 * (n // 64) for n in (T * D, T * F, T * F, T * F))


def test_block_shapes_are_checked():
    def q(N, K):
        return AdaptedLinear(api.NF4Weight(None, None, None, N, K))
    with pytest.raises(ValueError, match="do not form a block"):
        GatedMlp(q(128, 64), q(128, 64), q(128, 64))
    with pytest.raises(ValueError, match="act must be"):
        GatedMlp(q(128, 64), q(128, 64), q(64, 128), act="swish")
