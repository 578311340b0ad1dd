"""A gated feed-forward block from frozen-base linear layers: how the epilogue
forward, the 8-bit activation checkpoints and the backward from them run together.

    U = X Wu'^T + s (X Au) Bu
    H = silu(X Wg'^T + s (X Ag) Bg) * U          (the product in the gate's epilogue)
    Y = H Wd'^T + s (H Ad) Bd + residual         (the sum in the down projection's)

A training forward keeps X, the gate's pre-activation, U and H as checkpoints:
1.0625 bytes a value where 16-bit copies would take 2.  The backward reads them
and gives the gradients of X and of the three adapters; the residual's gradient
is dY itself.

``NormMlp`` puts the norm in front and the residual stream around the block,

    H = X + R,   Y = H + mlp(norm(H))

and ``Int8Mlp`` serves that block with its adapters merged: the norm writes 8-bit
rows, and all three products run on 8-bit integers.

The module only orders calls of ``api``; all arithmetic runs in the kernels.
"""
from dataclasses import dataclass

import torch

from . import api


@dataclass
class AdaptedLinear:
    """A frozen quantized weight and its adapter (None, None without one)."""
    qw: api.NF4Weight
    lora_a: torch.Tensor = None
    lora_b: torch.Tensor = None
    scaling: float = 1.0

    def args(self):
        return self.qw, self.lora_a, self.lora_b, self.scaling


@dataclass
class MlpSaved:
    """What a training forward keeps for the backward."""
    x: api.Act8
    z: api.Act8      # the gate's pre-activation
    u: api.Act8
    h: api.Act8

    def nbytes(self):
        return sum(a.nbytes() for a in (self.x, self.z, self.u, self.h))


@dataclass
class MlpGrads:
    dx: torch.Tensor
    gate: tuple      # (d_lora_a, d_lora_b), as are the others; (None, None) without an adapter
    up: tuple
    down: tuple


class GatedMlp:
    """Gate and up [F, D], down [D, F]; activation of the gate one of ``api.ACTS``."""

    def __init__(self, gate, up, down, act="silu"):
        D, F = gate.qw.K, gate.qw.N
        if (up.qw.N, up.qw.K) != (F, D) or (down.qw.N, down.qw.K) != (D, F):
            raise ValueError(f"gate [{F}, {D}], up [{up.qw.N}, {up.qw.K}] and down [{down.qw.N}, {down.qw.K}] "
                             "do not form a block")
        if act not in api.ACTS:
            raise ValueError(f"act must be one of {', '.join(api.ACTS)}, not {act!r}")
        self.gate, self.up, self.down, self.act = gate, up, down, act

    def forward(self, x, residual=None):
        """Y [T, D] of X [T, D] (prompts and single tokens alike)."""
        u = api.qlora_linear_act_fwd(x, *self.up.args())
        h = api.qlora_linear_act_fwd(x, *self.gate.args(), act=self.act, mul=u, out=u)
        return api.qlora_linear_act_fwd(h, *self.down.args(), residual=residual)

    def forward_train(self, x, residual=None):
        """(Y, MlpSaved)"""
        u = api.qlora_linear_act_fwd(x, *self.up.args())
        h, z8 = api.qlora_linear_act_fwd(x, *self.gate.args(), act=self.act, mul=u, save="z8")
        y = api.qlora_linear_act_fwd(h, *self.down.args(), residual=residual)
        return y, MlpSaved(api.act8_quantize(x), z8, api.act8_quantize(u), api.act8_quantize(h))

    def backward(self, dy, saved):
        """MlpGrads for the upstream gradient dY [T, D]."""
        def grads(layer):
            return layer.lora_a is not None
        d = api.qlora_linear_act_bwd(dy, *self.down.args(), x=saved.h, lora_grads=grads(self.down))
        g = api.qlora_linear_act_bwd(d.dx, *self.gate.args(), act=self.act, x=saved.x, z=saved.z, mul=saved.u,
                                     lora_grads=grads(self.gate))
        # both layers read X: their gradients are summed in the up projection's epilogue
        u = api.qlora_linear_act_bwd(g.d_mul, *self.up.args(), x=saved.x, lora_grads=grads(self.up), dx_add=g.dx,
                                     dx=g.dx)
        return MlpGrads(u.dx, (g.d_lora_a, g.d_lora_b), (u.d_lora_a, u.d_lora_b), (d.d_lora_a, d.d_lora_b))


@dataclass
class NormMlpSaved:
    """What a training forward keeps for the backward."""
    h: torch.Tensor      # the residual stream in front of the norm, 16 bits (x itself where nothing was added to it)
    mlp: MlpSaved

    def nbytes(self):
        return self.h.numel() * self.h.element_size() + self.mlp.nbytes()


@dataclass
class NormMlpGrads:
    dx: torch.Tensor      # of x and of residual alike
    d_norm: torch.Tensor  # of the norm's weight (None if it is frozen)
    mlp: MlpGrads


class NormMlp:
    """A GatedMlp behind a root-mean-square norm, with the residual stream around both.
    norm_weight [D] in the activations' dtype or float32, or None for ones."""

    def __init__(self, mlp, norm_weight=None, eps=1e-6):
        if norm_weight is not None and tuple(norm_weight.shape) != (mlp.gate.qw.K,):
            raise ValueError(f"norm_weight has shape {tuple(norm_weight.shape)}, expected {(mlp.gate.qw.K,)}")
        self.mlp, self.norm_weight, self.eps = mlp, norm_weight, eps

    def _normed(self, x, residual):
        if residual is None:
            return api.rmsnorm_fwd(x, self.norm_weight, self.eps), x
        return api.rmsnorm_fwd(x, self.norm_weight, self.eps, residual=residual)

    def forward(self, x, residual=None):
        """Y [T, D] of X [T, D] and what is added to it first (the attention's output, say)."""
        n, h = self._normed(x, residual)
        return self.mlp.forward(n, residual=h)

    def forward_train(self, x, residual=None):
        """(Y, NormMlpSaved)"""
        n, h = self._normed(x, residual)
        y, saved = self.mlp.forward_train(n, residual=h)
        return y, NormMlpSaved(h, saved)

    def backward(self, dy, saved, norm_grad=True):
        """NormMlpGrads for the upstream gradient dY [T, D] (its mlp.dx is the buffer that dx is formed in)."""
        m = self.mlp.backward(dy, saved.mlp)
        g = api.rmsnorm_bwd(m.dx, saved.h, self.norm_weight, self.eps, dx_add=dy, weight_grad=norm_grad, dx=m.dx)
        return NormMlpGrads(g.dx, g.d_weight, m)


class Int8Mlp:
    """A NormMlp for serving, its three weights (Rows8, one scale per output channel) as products of 8-bit
    integers: gate and up [F, D], down [D, F]."""

    def __init__(self, gate, up, down, norm_weight=None, eps=1e-6, act="silu"):
        F, D = gate.shape
        if up.shape != (F, D) or down.shape != (D, F):
            raise ValueError(f"gate {gate.shape}, up {up.shape} and down {down.shape} do not form a block")
        if act not in api.ACTS:
            raise ValueError(f"act must be one of {', '.join(api.ACTS)}, not {act!r}")
        self.gate, self.up, self.down = gate, up, down
        self.norm_weight, self.eps, self.act = norm_weight, eps, act

    @classmethod
    def from_block(cls, block, dtype=torch.bfloat16):
        """Of a NormMlp: every adapter merged into its weight (in the adapter's dtype; a weight without one is
        taken in `dtype`), the weight's rows quantized."""
        rows = (api.rows8_quantize(api.qlora_merge_lora(*layer.args(), dtype=dtype))
                for layer in (block.mlp.gate, block.mlp.up, block.mlp.down))
        return cls(*rows, block.norm_weight, block.eps, block.mlp.act)

    def forward(self, x, residual=None):
        """Y [T, D] of X [T, D] and what is added to it first (prompts and single tokens alike)."""
        n = api.rmsnorm_fwd(x, self.norm_weight, self.eps, residual=residual, quantize=True)
        n, h = (n, x) if residual is None else n
        u = api.int8_linear_fwd(n, self.up, dtype=x.dtype)
        u = api.int8_linear_fwd(n, self.gate, act=self.act, mul=u, out=u)
        return api.int8_linear_fwd(api.rows8_quantize(u), self.down, residual=h, dtype=x.dtype)
