"""Every kernel of the 8-bit product, at sizes that leave remainders in each direction, with
every epilogue; and the norm's backward where long rows are read past the caches.

An 8-bit product without an activation (or with relu) is a fixed sequence of fp32 operations,

    z = fl32(fl32(fl32(sum) min) max),  z = fl32(z + bias),  relu,  z = fl32(z mul),  z = fl32(z + residual)

rounded once to 16 bits: it is compared bit for bit.  With the other activations the same token
and channel give the same bits through every kernel; test_gpu_block.py holds them to the
oracle on the kernels of few tokens."""
import numpy as np
import pytest
import torch

import oracle
from qlora_linear_layers_amd import api
from helpers import say
from test_gpu_block import DT, TINY, U, behind, f64, make, rows8_of, within

# One row per kernel of the product, (T, N, K): the decode kernel with 16 and with 32 tokens a
# workgroup; tiles of 64 and 128 tokens, whole and with their reduction split (2 to 8 times);
# 128 x 128 tiles where they are several a CU (two LDS buffers); 256 x 256 tiles.
ROUTES = {
    "decode 16": [(1, 261, 300), (7, 100, 65), (16, 33, 2100)],
    "decode 32": [(17, 129, 300), (32, 257, 2050)],
    "64": [(64, 325, 128), (33, 66, 258)],
    "64 split": [(33, 11011, 1926), (34, 15, 1129), (33, 130, 1000), (36, 10, 1203), (43, 10, 1419), (35, 11, 1769),
                 (49, 9, 1983)],
    "128": [(130, 265, 384), (300, 513, 640)],
    "128 split": [(67, 11, 1044), (65, 9, 1291), (78, 10, 1275), (83, 10, 1478), (129, 300, 4099), (200, 29, 5001)],
    # 1 to 5 K tiles of 128: odd and even, fewer than and as many as the buffers and more
    "128 two buffers": [(1153, 3969, k) for k in (128, 130, 260, 400, 640)],
    "256": [(4000, 3001, k) for k in (128, 130, 260, 400, 640)],
}
ALL = [(r, *s) for r, shapes in ROUTES.items() for s in shapes]


def up(a, b):
    return -(-a // b)


def plan(T, K, N):
    """(kernel, splits) by the rules stated beside the kernels."""
    if T <= 16:
        return "decode 16", 1
    if T <= 32 and N <= 4096 and T * K <= 196608:
        return "decode 32", 1
    if 768 * up(up(N, 256) * up(T, 256), 256) <= up(N, 128) * up(T, 128):
        return "256", 1
    rows = 64 if T <= 64 else 128
    tiles, kt, splits = up(N, 128) * up(T, rows), up(K, 128), 1

    def cost(s):
        return up(tiles * s, 256) * up(kt, s) * 0.34 + (1.5 + 0.4e-6 * (s * T * N * 4) if s > 1 else 0.0)
    for s in range(2, 9):
        if kt // s < 2 or tiles * s > 256:
            break
        if cost(s) < cost(splits):
            splits = s
    if splits > 1:
        return f"{rows} split", splits
    return ("64" if rows == 64 else "128 two buffers" if tiles > 256 else "128"), 1


def test_the_sizes_reach_every_kernel():
    """The rules as restated here give the workspaces that the library asks for, and every kernel and
    every number of splits has a size above."""
    try:
        workspace = api.int8_linear_workspace_bytes
        workspace(1, 1, 1)
    except RuntimeError:
        pytest.skip("library not built")
    seen = set()
    for route, T, N, K in ALL:
        assert plan(T, K, N)[0] == route, (T, N, K)
        seen.add(plan(T, K, N))
    for kernel in ROUTES:
        assert any(k == kernel for k, _ in seen)
    assert {s for k, s in seen if k == "64 split"} | {s for k, s in seen if k == "128 split"} == set(range(2, 9))
    rng = np.random.default_rng(0)
    sizes = [(T, K, N) for _, T, N, K in ALL] + [tuple(int(2 ** v) for v in rng.uniform((0, 0, 0), (13, 14, 15)))
                                                for _ in range(3000)]
    for T, K, N in sizes:
        splits = plan(T, K, N)[1]
        need = splits * T * up(N, 8) * 32 if splits > 1 else 0
        assert workspace(T, K, N) == up(need, 256) * 256, (T, K, N)


def operands(seed, T, N, dt):
    """bias, mul and residual, made where they are used."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(sh, generator=g, device="cuda").to(dt) for sh in ((N,), (T, N), (T, N))]


def product(x8, w8):
    """fl32(fl32(fl32(sum) min) max) of every output, by torch's own operations (the sum is exact in fp64)."""
    s = (x8.codes.double() @ w8.codes.double().t().contiguous()).float()
    a, b = x8.scale[:, None], w8.scale[None, :]
    return s * torch.minimum(a, b) * torch.maximum(a, b)


def stepwise(x8, w8, dt, bias, act, mul, res):
    z = product(x8, w8)
    if bias is not None:
        z = z + bias.float()
    if act == "relu":
        z = torch.where(z <= 0, 0.0, z)
    if mul is not None:
        z = z * mul.float()
    if res is not None:
        z = z + res.float()
    return z.to(dt)


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("route,T,N,K", ALL)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_product_is_the_stated_operations(route, T, N, K, dtype):
    """Bit for bit, with every combination of bias, mul and residual; Y also in place of either."""
    n, dt = make(T + N + K), DT[dtype]
    x8, w8 = rows8_of(n, T, K), rows8_of(n, N, K, std=2 * K ** -0.5)
    b, m, r = operands(T + N + K, T, N, dt)
    for bias, mul, res, act in ((None, None, None, "none"), (b, None, None, "none"), (None, m, None, "relu"),
                                (None, None, r, "none"), (b, None, r, "relu"), (None, m, r, "none"), (b, m, r, "relu"),
                                (b, m, r, "none")):
        what = f"{route} T={T} N={N} K={K} {dtype} bias={bias is not None} mul={mul is not None} " \
               f"res={res is not None} {act}"
        say("[int8 routes] " + what)
        y, y_ok = behind(T, N, dt)
        api.int8_linear_fwd(x8, w8, bias=bias, act=act, mul=mul, residual=res, out=y)
        ref = stepwise(x8, w8, dt, bias, act, mul, res)
        assert same(y, ref), what
        assert y_ok(), what
        if mul is not None:
            t = mul.clone()
            assert same(api.int8_linear_fwd(x8, w8, bias=bias, act=act, mul=t, residual=res, out=t), ref), what
        if res is not None:
            t = res.clone()
            assert same(api.int8_linear_fwd(x8, w8, bias=bias, act=act, mul=mul, residual=t, out=t), ref), what


@pytest.mark.gpu
@pytest.mark.parametrize("route,T,N,K", [(r, *s[-1]) for r, s in ROUTES.items()])
@pytest.mark.parametrize("act", oracle.ACTS)
@pytest.mark.parametrize("dtype,bias,mul,res", [("bf16", True, False, False), ("fp16", True, True, True),
                                                ("bf16", False, True, True), ("fp16", False, False, True)])
def test_every_kernel_gives_a_token_the_same_bits(route, T, N, K, act, dtype, bias, mul, res):
    """Rows of a large product against the decode kernel's for the same tokens, and columns against
    those of a product of fewer channels (whose last are not a whole eight)."""
    say(f"[int8 routes] {route} T={T} N={N} K={K} {act} {dtype} bias={bias} mul={mul} res={res}")
    n, dt = make(T + N + K), DT[dtype]
    x8, w8 = rows8_of(n, T, K), rows8_of(n, N, K, std=2 * K ** -0.5)
    b, m, r = (t if on else None for t, on in zip(operands(T + N + K, T, N, dt), (bias, mul, res)))
    y = api.int8_linear_fwd(x8, w8, dtype=dt, bias=b, act=act, mul=m, residual=r)

    def part(rows, cols):
        cut = lambda t: None if t is None else t[rows, cols].clone()
        xs = x8.codes[rows].clone()
        ws = w8.codes[cols].clone()
        return api.int8_linear_fwd(api.Rows8(xs, x8.scale[rows].clone(), (xs.shape[0], K)),
                                   api.Rows8(ws, w8.scale[cols].clone(), (ws.shape[0], K)), dtype=dt,
                                   bias=None if b is None else b[cols].clone(), act=act, mul=cut(m), residual=cut(r))
    for lo, hi in ((0, 1), (0, min(T, 16)), (T // 2, min(T, T // 2 + 5)), (max(0, T - 16), T), (max(0, T - 40), T)):
        rows, cols = slice(lo, hi), slice(0, N)
        assert same(part(rows, cols), y[rows]), (lo, hi)
    for cols in (slice(0, max(1, N // 2 - 3)), slice(N // 3, N), slice(N - 1, N)):
        assert same(part(slice(0, T), cols), y[:, cols].contiguous()), cols


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", [s for r in ("64 split", "128 split") for s in ROUTES[r]])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_epilogue_of_split_products(T, N, K, act, dtype):
    """Against the oracle, with the bound of test_gpu_block.py."""
    say(f"[int8 routes] epilogue of splits T={T} N={N} K={K} {act} {dtype}")
    n, dt = make(T + N + K), DT[dtype]
    x8, w8 = rows8_of(n, T, K), rows8_of(n, N, K, std=2 * K ** -0.5)
    b, m, r = operands(T + N + K, T, N, dt)
    y, y_ok = behind(T, N, dt)
    api.int8_linear_fwd(x8, w8, bias=b, act=act, mul=m, residual=r, out=y)
    torch.cuda.synchronize()
    assert y_ok()
    ry, rz = oracle.int8_linear(x8.codes.cpu().numpy(), f64(x8.scale), w8.codes.cpu().numpy(), f64(w8.scale), f64(b), act,
                                f64(m), f64(r))
    mag = np.abs(rz) + np.abs(oracle.act(rz, act)) + np.abs(f64(b))
    within(y, ry, U[dt] * np.abs(ry) + 2e-5 * mag * np.abs(f64(m)) + 2.0 ** -23 * np.abs(f64(r)) + TINY[dt], "y")


# Rows of 8193 .. 12288 values (512 threads of three chunks), and batches that pass by the caches with dx_add (256 MiB
# at 8 bytes a value) and without (6 bytes)
@pytest.mark.gpu
@pytest.mark.parametrize("T,D,dtype", [(4099, 8456, "bf16"), (3001, 12288, "fp16"), (4099, 8200, "fp16"),
                                       (3600, 11008, "bf16"), (3001, 11999, "bf16"), (5500, 8200, "bf16"),
                                       (43711, 1032, "fp16"), (10950, 4088, "bf16")])
@pytest.mark.parametrize("add", [True, False])
def test_norm_backward_of_long_rows_in_large_batches(T, D, dtype, add):
    say(f"[norm backward, large] {T} x {D} {dtype} add={add}")
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(T + D)
    dy, h, ad = (torch.randn((T, D), generator=g, device="cuda").to(dt) for _ in range(3))
    w = torch.randn(D, generator=g, device="cuda")
    cut = lambda lo, hi: ad[lo:hi].clone() if add else None
    got = api.rmsnorm_bwd(dy, h, w, 1e-5, dx_add=ad if add else None)
    frozen = api.rmsnorm_bwd(dy, h, w, 1e-5, dx_add=ad if add else None, weight_grad=False)
    assert same(got.dx, frozen.dx)
    for lo, hi in ((0, 9), (T // 2, T // 2 + 5), (T - 7, T)):
        few = api.rmsnorm_bwd(dy[lo:hi].clone(), h[lo:hi].clone(), w, 1e-5, dx_add=cut(lo, hi))
        assert same(got.dx[lo:hi], few.dx), (lo, hi)
    ref, size = (torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(2))
    for lo in range(0, T, 1024):
        hd = h[lo:lo + 1024].double()
        terms = dy[lo:lo + 1024].double() * hd * (hd.square().mean(1, keepdim=True) + 1e-5).rsqrt()
        ref += terms.sum(0)
        size += terms.abs().sum(0)
    within(got.d_weight, f64(ref), U[torch.float32] * np.abs(f64(ref)) + 1e-5 * f64(size), "dw")
