"""The pre-norm block (NormMlp) and its 8-bit serving form (Int8Mlp) against the fp64
oracle composed the same way.

Tolerances, u the half step of the 16-bit type.  The training block adds to GatedMlp's
roundings (at most 2 u forward, 2.5 u backward relative to the branch, as derived for it)
the rounding of the normed input, at most u / sqrt(3) carried by products that average it:
3 u forward.  Backward, dX is the branch's gradient through the norm plus dY: the branch's
2.5 u, one more rounding (d mlp / d n) and the last: 4 u.  The norm's weight gradient sums the branch's
gradient: 4 u.  What checkpoints cost is left out by differentiating at the values they
stand for.  8 bits: one code is off by half a unit of max / 127.  With normal values max is
about 3.7 rms of 256 to 448, the normed rows' and weights' codes are each off by
3.7 / 127 / sqrt(12) = 0.84% of the rms, the hidden rows' (products of two normals, max about 8
rms) by 1.9%; the branch sees the first two through up and gate each and the last two
through down: sqrt(0.84^2 x 2 x 2 + 1.9^2 + 0.84^2) = 2.7%, so below 4%."""
import numpy as np
import pytest
import torch

import oracle
from qlora_linear_layers_amd import api
from qlora_linear_layers_amd.mlp import AdaptedLinear, GatedMlp, Int8Mlp, NormMlp
from helpers import say

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _rel(got, ref, scale=None):
    return float(np.linalg.norm(_f64(got) - ref) / np.linalg.norm(ref if scale is None else scale))


def _block(D, F, r, dt, w32, seed=0):
    g = torch.Generator().manual_seed(D + F + seed)
    n = lambda *sh, std=1.0, dt=dt: (torch.randn(sh, generator=g) * std).to(dt).cuda()

    def linear(N, K):
        qw = api.nf4_quantize_dq(n(N, K, std=1.0 / K ** 0.5))
        return AdaptedLinear(qw, n(K, r, std=0.05), n(r, N, std=0.2), 0.5) if r else AdaptedLinear(qw)
    mlp = GatedMlp(linear(F, D), linear(F, D), linear(D, F))
    w = (1 + 0.2 * n(D, dt=torch.float32)).to(torch.float32 if w32 else dt)
    return n, NormMlp(mlp, w, 1e-5)


def _weights(block, dt):
    def one(l):
        a, b = (_f64(l.lora_a), _f64(l.lora_b)) if l.lora_a is not None else (None, None)
        return _f64(api.nf4_dequantize_dq(l.qw, dtype=dt)), a, b
    return [one(l) for l in (block.mlp.gate, block.mlp.up, block.mlp.down)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,F,r,dt,res", [(1, 256, 320, 8, torch.bfloat16, True), (40, 320, 192, 0, torch.bfloat16, False),
                                            (300, 256, 448, 24, torch.bfloat16, True),
                                            (130, 256, 448, 16, torch.float16, True)])
def test_norm_block_matches_the_oracle(T, D, F, r, dt, res):
    say(f"[norm mlp] T={T} D={D} F={F} r={r} {dt} residual={res}")
    n, block = _block(D, F, r, dt, w32=dt == torch.bfloat16)
    s, u, eps = 0.5, U[dt], 1e-5
    x, dy = n(T, D), n(T, D)
    rs = n(T, D) if res else None
    y, saved = block.forward_train(x, rs)
    grads = block.backward(dy, saved)
    frozen = block.backward(dy, saved, norm_grad=False)
    torch.cuda.synchronize()
    assert torch.equal(block.forward(x, rs), y)
    assert frozen.d_norm is None and torch.equal(frozen.dx, grads.dx)
    assert grads.d_norm.dtype == block.norm_weight.dtype and saved.nbytes() == T * D * 2 + saved.mlp.nbytes()

    wg, wu, wd = _weights(block, dt)
    w, h = _f64(block.norm_weight), _f64(saved.h)
    rn = oracle.rmsnorm(h, w, eps)
    ru = oracle.act_fwd(rn, *wu, s)[0]
    rh = oracle.act_fwd(rn, *wg, s, name="silu", mul=ru)[0]
    ry = oracle.act_fwd(rh, *wd, s, residual=h)[0]
    e = _rel(y, ry)
    say(f"  Y: {e / u:.2f} u")
    assert e < 3 * u
    value = lambda a: oracle.ck_values(a.codes.cpu().numpy(), a.scale.cpu().numpy()).reshape(a.shape)
    m = saved.mlp
    d = oracle.act_bwd(_f64(dy), *wd, s, x=value(m.h))
    gg = oracle.act_bwd(d["dx"], *wg, s, "silu", x=value(m.x), z=value(m.z), mul=value(m.u))
    dn = oracle.act_bwd(gg["dmul"], *wu, s, x=value(m.x), dx_add=gg["dx"])["dx"]
    rdx, rdw = oracle.rmsnorm_bwd(dn, h, w, eps, _f64(dy))
    for name, got, ref in (("dX", grads.dx, rdx), ("d norm", grads.d_norm, rdw)):
        e = _rel(got, ref)
        say(f"  {name}: {e / u:.2f} u")
        assert e < 4 * u, name


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 9, 40, 300])
@pytest.mark.parametrize("dt,res", [(torch.bfloat16, True), (torch.float16, False)])
def test_int8_block_matches_the_merged_one(T, dt, res):
    say(f"[int8 mlp] T={T} {dt} residual={res}")
    D, F, s = 256, 448, 0.5
    n, block = _block(D, F, 16, dt, w32=False, seed=1)
    served = Int8Mlp.from_block(block, dtype=dt)
    x, rs = n(T, D), n(T, D) if res else None
    y = served.forward(x, rs)
    torch.cuda.synchronize()
    assert y.dtype == dt
    (wg, ag, bg), (wu, au, bu), (wd, ad, bd) = _weights(block, dt)
    wg, wu, wd = wg + s * (ag @ bg).T, wu + s * (au @ bu).T, wd + s * (ad @ bd).T
    h = _f64(x) if rs is None else _f64((x.float() + rs.float()).to(dt))
    rn = oracle.rmsnorm(h, _f64(block.norm_weight), 1e-5)
    hidden = oracle.act(rn @ wg.T, "silu") * (rn @ wu.T)
    branch = hidden @ wd.T
    e = float(np.linalg.norm(_f64(y) - h - branch) / np.linalg.norm(branch))
    say(f"  branch off by {e:.4f}")
    assert e < 0.04


def test_block_shapes_are_checked():
    def q(N, K):
        return AdaptedLinear(api.NF4Weight(None, None, None, N, K))
    mlp = GatedMlp(q(128, 64), q(128, 64), q(64, 128))
    with pytest.raises(ValueError, match="norm_weight has shape"):
        NormMlp(mlp, torch.ones(128))
    r = lambda N, K: api.Rows8(None, None, (N, K))
    with pytest.raises(ValueError, match="do not form a block"):
        Int8Mlp(r(128, 64), r(128, 64), r(128, 64))
    with pytest.raises(ValueError, match="act must be"):
        Int8Mlp(r(128, 64), r(128, 64), r(64, 128), act="swish")
