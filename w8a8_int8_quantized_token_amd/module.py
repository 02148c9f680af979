"""Drop-in modules: a bf16 nn.Linear, a gated feed-forward block and a QKV
projection with normed and rotated queries and keys, with the weights quantized
once per output channel and the activations per token on every call.

The weights are frozen codes; gradients pass through to the input (and to the
norm weights of the QKV projection)."""
from __future__ import annotations

import torch

from . import autograd, block_ops, ops


def _codes(*linears: torch.nn.Linear):
    """Codes, scales and bias of one or more linears, one below the other."""
    parts = [ops.quantize_weight(l.weight.detach().to(torch.bfloat16).contiguous()) for l in linears]
    biases = [l.bias for l in linears]
    if any(b is None for b in biases) and not all(b is None for b in biases):
        raise ValueError("either every linear has a bias or none")
    bias = None if biases[0] is None else torch.cat([b.detach().to(torch.bfloat16) for b in biases])
    if len(parts) == 1:
        return (*parts[0], bias)
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts]), bias


def _tokens(x: torch.Tensor, features: int, name: str) -> torch.Tensor:
    x2 = x.reshape(-1, features)
    if x2.dtype != torch.bfloat16:
        raise TypeError(f"{name} expects bf16 activations")
    return x2.contiguous()


class W8A8Linear(torch.nn.Module):
    def __init__(self, wq: torch.Tensor, w_scale: torch.Tensor, bias: torch.Tensor | None):
        super().__init__()
        self.register_buffer("wq", wq)
        self.register_buffer("w_scale", w_scale)
        self.register_buffer("bias", bias)
        self.out_features, self.in_features = wq.shape

    @classmethod
    def from_linear(cls, lin: torch.nn.Linear) -> "W8A8Linear":
        return cls(*_codes(lin))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        lead = x.shape[:-1]
        x2 = _tokens(x, self.in_features, "W8A8Linear")
        if x2.requires_grad and torch.is_grad_enabled():
            y = autograd._FrozenLinear.apply(x2, self.wq, self.w_scale, self.bias)
        else:
            y = block_ops.linear_dynamic(x2, self.wq, self.w_scale, self.bias)
        return y.reshape(*lead, self.out_features)


class W8A8GatedMLP(torch.nn.Module):
    """down(act(gate(x)) * up(x)): the gate and up projections, the activation
    and the product in one kernel, then the down projection."""

    def __init__(self, wq: torch.Tensor, w_scale: torch.Tensor, bias: torch.Tensor | None, down: W8A8Linear,
                 act: str = "silu"):
        super().__init__()
        if wq.shape[0] != 2 * down.in_features:
            raise ValueError("gate and up must each have as many channels as down has inputs")
        block_ops._act(act)
        self.register_buffer("wq", wq)
        self.register_buffer("w_scale", w_scale)
        self.register_buffer("bias", bias)
        self.down, self.act = down, act
        self.in_features = wq.shape[1]

    @classmethod
    def from_linears(cls, gate: torch.nn.Linear, up: torch.nn.Linear, down: torch.nn.Linear,
                     act: str = "silu") -> "W8A8GatedMLP":
        if gate.weight.shape != up.weight.shape:
            raise ValueError("gate and up must have the same shape")
        return cls(*_codes(gate, up), W8A8Linear.from_linear(down), act)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        x2 = _tokens(x, self.in_features, "W8A8GatedMLP")
        if x2.requires_grad and torch.is_grad_enabled():
            h = autograd._Gated.apply(x2, self.wq, self.w_scale, self.bias, self.act)
        else:
            h = block_ops.gated_linear_dynamic(x2, self.wq, self.w_scale, self.bias, act=self.act)
        return self.down(h).reshape(*x.shape[:-1], self.down.out_features)


class W8A8QKV(torch.nn.Module):
    """The QKV projection of an attention block, with the RMS norm of each
    query and key head and the position rotation.  The projection's rows are
    Hq query heads, Hk key heads and Hk value heads of D channels."""

    def __init__(self, proj: W8A8Linear, q_heads: int, k_heads: int, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False):
        super().__init__()
        heads = q_heads + 2 * k_heads
        if proj.out_features % heads:
            raise ValueError("the projection's rows are not whole heads")
        self.proj, self.eps, self.interleaved = proj, eps, interleaved
        self.heads = (q_heads, k_heads, proj.out_features // heads)
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            self.register_parameter(name, None if w is None else
                                    torch.nn.Parameter(w.detach().to(torch.bfloat16).contiguous()))

    @staticmethod
    def _tables(tokens: int, sequences: int, cos: torch.Tensor, sin: torch.Tensor):
        """The tables cut to the sequences' length, so that row mod P of the
        flattened batch is the index in a sequence."""
        if any(not isinstance(t, torch.Tensor) or t.dim() != 2 for t in (cos, sin)) or cos.shape != sin.shape or \
                cos.numel() == 0:
            return cos, sin     # what is wrong is named by the call, and without a rotation there are no positions
        P = cos.shape[0]
        if sequences > 1 and tokens > P and tokens % P:
            raise ValueError(f"sequences of {tokens} tokens are no whole runs of the {P} positions of cos and sin: "
                             "give each token's position")
        if 0 < tokens < P:
            return cos[:tokens], sin[:tokens]
        return cos, sin

    def forward(self, x: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, positions: torch.Tensor | None = None):
        """x [..., features] -> q [..., Hq, D], k and v [..., Hk, D]; cos, sin
        fp32 [P, rot/2], positions int32, one per token.  Without positions a
        token is at its index in its sequence (the last dimension before the
        features), in sequences longer than the tables at that index mod P."""
        if positions is None and x.dim() > 2:
            cos, sin = self._tables(x.shape[-2], x.shape[:-2].numel(), cos, sin)
        qkv = self.proj(x).reshape(-1, self.proj.out_features)
        if positions is not None:
            positions = positions.reshape(-1)
        grads = torch.is_grad_enabled() and any(
            t is not None and t.requires_grad for t in (qkv, self.q_weight, self.k_weight))
        if grads:
            q, k, v = autograd._QKNormRope.apply(qkv, self.q_weight, self.k_weight, cos, sin, positions, self.heads,
                                                 self.eps, self.interleaved)
        else:
            q, k, v = autograd._split(qkv, self.heads)
            # not in place: a hook on the projection may keep its output
            q, k = block_ops.qk_norm_rope(q, k, self.q_weight, self.k_weight, cos, sin, positions, self.eps,
                                          self.interleaved)
        lead = x.shape[:-1]
        return tuple(t.reshape(*lead, *t.shape[1:]) for t in (q, k, v))
