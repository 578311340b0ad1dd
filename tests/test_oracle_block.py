"""Pins of the norm, the 8-bit rows and the 8-bit product in the oracle: closed
forms, differences, torch's own norm, brute force."""
import numpy as np
import pytest
import torch

import oracle


def test_rows8_closed_forms():
    x = np.array([[127.0, -64.0, 0.5, 1.5, -2.5], [0, 0, 0, 0, 0], [2.0 ** -121, 0, 0, 0, 0],
                  [1.0, np.inf, 0, 0, 0], [1.0, np.nan, 0, 0, 0], [-254.0, 1.0, 3.0, 5.0, 253.0]])
    q, d = oracle.rows8_quantize(x)
    assert q.shape == (6, 128) and not q[:, 5:].any()
    # row 0: unit 1, halves to even; row 5: unit 2
    assert q[0, :5].tolist() == [127, -64, 0, 2, -2] and d[0] == 1.0
    assert q[5, :5].tolist() == [-127, 0, 2, 2, 126] and d[5] == 2.0
    assert not q[1:5].any() and d[1] == 0 and d[2] == 0 and np.isnan(d[3]) and np.isnan(d[4])
    v = oracle.rows8_values(q, d, 5)
    assert np.array_equal(v[5], [-254.0, 0, 4, 4, 252]) and np.isnan(v[3]).all()


@pytest.mark.parametrize("K", [1, 64, 127, 300])
def test_rows8_is_within_half_a_unit(K):
    x = np.random.default_rng(K).standard_normal((9, K)).astype(np.float32).astype(np.float64)
    q, d = oracle.rows8_quantize(x)
    assert np.abs(q[:, :K]).max(1).tolist() == [127] * 9
    # half a unit, the factor's rounding on top (127 codes times 2^-23)
    assert (np.abs(oracle.rows8_values(q, d, K) - x) <= d[:, None] * (0.5 + 127 * 2.0 ** -22)).all()


def test_norm_is_torchs():
    g = np.random.default_rng(0)
    h, w = g.standard_normal((5, 37)), g.standard_normal(37)
    eps = float(np.float32(1e-5))
    ref = torch.nn.functional.rms_norm(torch.from_numpy(h), (37,), torch.from_numpy(w), eps).numpy()
    assert np.allclose(oracle.rmsnorm(h, w, 1e-5), ref, rtol=1e-13, atol=0)


def test_norm_gradient_against_autograd_and_differences():
    g = np.random.default_rng(1)
    h, w, dy, add = g.standard_normal((4, 11)), g.standard_normal(11), g.standard_normal((4, 11)), g.standard_normal((4, 11))
    dx, dw = oracle.rmsnorm_bwd(dy, h, w, 1e-3, add)
    th, tw = torch.from_numpy(h).requires_grad_(), torch.from_numpy(w).requires_grad_()
    y = torch.nn.functional.rms_norm(th, (11,), tw, float(np.float32(1e-3)))
    a, b = torch.autograd.grad(y, (th, tw), torch.from_numpy(dy))
    assert np.allclose(dx, a.numpy() + add, rtol=1e-12) and np.allclose(dw, b.numpy(), rtol=1e-12)
    step = 1e-6
    for i, j in ((0, 0), (2, 7), (3, 10)):
        e = np.zeros_like(h)
        e[i, j] = step
        diff = ((oracle.rmsnorm(h + e, w, 1e-3) - oracle.rmsnorm(h - e, w, 1e-3)) * dy).sum() / (2 * step)
        assert abs(diff - (dx - add)[i, j]) < 1e-8
    assert oracle.rmsnorm_bwd(dy, h, None, 1e-3)[1] is None


def test_int8_linear_brute_force():
    g = np.random.default_rng(2)
    xq, wq = (g.integers(-127, 128, s).astype(np.int8) for s in ((3, 40), (5, 40)))
    xs, ws, bias = g.random(3).astype(np.float32), g.random(5).astype(np.float32), g.standard_normal(5)
    mul, res = g.standard_normal((3, 5)), g.standard_normal((3, 5))
    y, z = oracle.int8_linear(xq, xs, wq, ws, bias, "relu", mul, res)
    for t in range(3):
        for n in range(5):
            s = sum(int(a) * int(b) for a, b in zip(xq[t], wq[n]))
            zz = s * float(xs[t]) * float(ws[n]) + bias[n]
            assert abs(z[t, n] - zz) < 1e-9 and abs(y[t, n] - (max(zz, 0.0) * mul[t, n] + res[t, n])) < 1e-9
