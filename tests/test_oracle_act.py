"""Pins of the activation and checkpoint oracle: slopes against differences, the
backward against differences of the forward, known values, and the checkpoint's
bounds and edge blocks."""
import numpy as np
import pytest

import oracle


def test_known_values():
    z = np.array([-1.0, 0.0, 1.0, 3.0])
    assert np.allclose(oracle.act(z, "silu"), [-0.2689414213699951, 0.0, 0.7310585786300049, 2.8577223804673])
    assert np.allclose(oracle.act(z, "gelu"), [-0.15865525393145707, 0.0, 0.8413447460685429, 2.9959503059])
    assert np.allclose(oracle.act(z, "gelu_tanh"), oracle.act(z, "gelu"), atol=5e-4)
    assert np.array_equal(oracle.act(z, "relu"), [0.0, 0.0, 1.0, 3.0])


@pytest.mark.parametrize("name", oracle.ACTS)
def test_slopes_are_the_derivatives(name):
    z = np.linspace(-9.0, 9.0, 4001) + 1e-4              # off relu's corner
    e = 1e-5
    diff = (oracle.act(z + e, name) - oracle.act(z - e, name)) / (2 * e)
    # central difference: e^2/6 |act'''| (< 1e-10) and 2^-52 |z| / e (< 3e-10)
    assert np.max(np.abs(diff - oracle.act_slope(z, name))) < 1e-9
    far = np.array([-1e30, -300.0, 300.0, 1e30])
    with np.errstate(all="ignore"):
        assert np.allclose(oracle.act_slope(far[1:3], name), {"none": [1, 1]}.get(name, [0, 1]))


@pytest.mark.parametrize("name", oracle.ACTS)
@pytest.mark.parametrize("with_mul", [False, True])
def test_backward_is_the_derivative_of_the_forward(name, with_mul):
    g = np.random.default_rng(5)
    T, K, N, r, s = 5, 7, 6, 3, 0.5
    p = dict(x=g.standard_normal((T, K)), a=g.standard_normal((K, r)), b=g.standard_normal((r, N)),
             bias=g.standard_normal(N), mul=g.standard_normal((T, N)))
    w, dy = g.standard_normal((N, K)), g.standard_normal((T, N))

    def loss(q):
        y, z = oracle.act_fwd(q["x"], w, q["a"], q["b"], s, q["bias"], name, q["mul"] if with_mul else None)
        return float((y * dy).sum()), z
    z = loss(p)[1]
    got = oracle.act_bwd(dy, w, p["a"], p["b"], s, name, p["x"], z, p["mul"] if with_mul else None)
    for var, grad in (("x", "dx"), ("a", "da"), ("b", "db"), ("bias", "dbias")) + ((("mul", "dmul"),) if with_mul else ()):
        v = g.standard_normal(p[var].shape)
        e = 1e-6
        d = (loss({**p, var: p[var] + e * v})[0] - loss({**p, var: p[var] - e * v})[0]) / (2 * e)
        # |loss| < 1e3: 2^-52 1e3 / 1e-6 = 2e-7 of cancellation
        assert abs(d - float((got[grad] * v).sum())) < 1e-5, grad


def test_checkpoint_bounds_and_edge_blocks():
    g = np.random.default_rng(1)
    x = oracle.bf16_bits_to_f64(oracle.round_to_bf16_bits(g.standard_normal(64 * 5 + 9) * 3))
    x[64:128] = 0.0
    x[128:192] *= 2.0 ** -125
    x = oracle.bf16_bits_to_f64(oracle.round_to_bf16_bits(x))
    q, d = oracle.ck_quantize(x)
    assert q.shape == x.shape and d.shape == (6,)
    assert np.all(q[64:192] == 0) and np.all(d[1:3] == 0)
    v = oracle.ck_values(q, d)
    for b in (0, 3, 4, 5):
        s = slice(64 * b, 64 * b + 64)
        assert abs(int(np.abs(q[s].astype(int)).max())) == 127
        assert np.max(np.abs(v[s] - x[s])) <= float(d[b]) * (0.5 + 127 * 2.0 ** -23)
    y = x.copy()
    y[3], y[70] = np.inf, np.nan
    q, d = oracle.ck_quantize(y)
    assert np.isnan(d[0]) and np.isnan(d[1]) and np.all(q[:128] == 0) and np.isfinite(d[2:]).all()
    # half way between two codes (c = 254, unit 2): to the even one
    t = np.zeros(64)
    t[:5] = [254.0, 127.0, 1.0, 3.0, -5.0]
    assert list(oracle.ck_quantize(t)[0][:5]) == [127, 64, 0, 2, -2]
