"""A gated feed-forward block from frozen-base linear layers: how the epilogue
forward, the 8-bit activation checkpoints and the backward from them run together.

    U = X Wu'^T + s (X Au) Bu
    H = silu(X Wg'^T + s (X Ag) Bg) * U          (the product in the gate's epilogue)
    Y = H Wd'^T + s (H Ad) Bd + residual         (the sum in the down projection's)

A training forward keeps X, the gate's pre-activation, U and H as checkpoints:
1.0625 bytes a value where 16-bit copies would take 2.  The backward reads them
and gives the gradients of X and of the three adapters; the residual's gradient
is dY itself.

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
