"""Drop-in modules: a bf16 nn.Linear, a gated feed-forward block and a QKV
projection with normed and rotated queries and keys, with the weights quantized
once per output channel and the activations per token on every call.

The weights are frozen codes; gradients pass through to the input (and to the
norm weights of the QKV projection, and to low-rank adapters beside a linear).
A norm in front of a linear leaves the activations' codes, which the modules
take in the place of bf16 activations."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import adapter_ops, autograd, block_ops, ops


class Tokens(NamedTuple):
    """Activations as codes: int8 [..., K], one fp32 scale per token [...], and
    the codes' stand-in for gradients (bf16 [..., K] without memory of its own,
    or None)."""

    codes: torch.Tensor
    scale: torch.Tensor
    stand_in: torch.Tensor | None = None

    @property
    def shape(self) -> torch.Size:
        return self.codes.shape

    def dim(self) -> int:
        return self.codes.dim()


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


def _tokens(x: torch.Tensor | Tokens, features: int, name: str):
    """x as rows: bf16 [M, features], or Tokens of as many."""
    if isinstance(x, Tokens):
        if x.codes.shape[-1] != features or x.scale.shape != x.codes.shape[:-1]:
            raise ValueError(f"{name} expects codes of {features} features with one scale per token")
        stand_in = x.stand_in
        if stand_in is not None:
            stand_in = stand_in.reshape(-1, features) if stand_in.requires_grad and torch.is_grad_enabled() else None
        return Tokens(x.codes.reshape(-1, features).contiguous(), x.scale.reshape(-1).contiguous(), stand_in)
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

    def forward(self, x: torch.Tensor | Tokens) -> torch.Tensor:
        lead = x.shape[:-1]
        x2 = _tokens(x, self.in_features, "W8A8Linear")
        if isinstance(x2, Tokens):
            if x2.stand_in is not None:
                y = autograd._CodesLinear.apply(x2.stand_in, x2.codes, x2.scale, self.wq, self.w_scale, self.bias)
            else:
                with torch.cuda.device_of(x2.codes):
                    y = ops.linear(x2.codes, x2.scale, self.wq, self.w_scale, self.bias)
        elif x2.requires_grad and torch.is_grad_enabled():
            y = autograd._FrozenLinear.apply(x2, self.wq, self.w_scale, self.bias)
        else:
            y = block_ops.linear_dynamic(x2, self.wq, self.w_scale, self.bias)
        return y.reshape(*lead, self.out_features)


class W8A8AdaptedLinear(W8A8Linear):
    """W8A8Linear with a set of low-rank adapters beside the frozen weight:
    a [L,R,K], b [L,N,R] (trainable) and scaling [L]; each token is assigned
    one of them, or none."""

    def __init__(self, wq: torch.Tensor, w_scale: torch.Tensor, bias: torch.Tensor | None, a: torch.Tensor,
                 b: torch.Tensor, scaling: torch.Tensor):
        super().__init__(wq, w_scale, bias)
        L, R = a.shape[:2]
        if a.shape != (L, R, self.in_features) or b.shape != (L, self.out_features, R) or scaling.shape != (L,):
            raise ValueError("a must be [adapters, rank, inputs], b [adapters, outputs, rank], scaling [adapters]")
        self.a = torch.nn.Parameter(a.detach().to(torch.bfloat16).contiguous())
        self.b = torch.nn.Parameter(b.detach().to(torch.bfloat16).contiguous())
        self.register_buffer("scaling", scaling.detach().to(torch.float32).contiguous())

    @classmethod
    def from_linear(cls, lin: torch.nn.Linear | W8A8Linear, adapters: int = 1, rank: int = 16,
                    scaling: float = 1.0) -> "W8A8AdaptedLinear":
        """New adapters that change nothing yet (b zeros) beside a linear."""
        wq, w_scale, bias = (lin.wq, lin.w_scale, lin.bias) if isinstance(lin, W8A8Linear) else _codes(lin)
        (N, K), dev = wq.shape, wq.device
        a = torch.randn(adapters, rank, K, device=dev) / K ** 0.5
        return cls(wq, w_scale, bias, a, torch.zeros(adapters, N, rank, device=dev),
                   torch.full((adapters,), float(scaling), device=dev))

    def forward(self, x: torch.Tensor | Tokens, adapters: torch.Tensor | int = 0) -> torch.Tensor:
        """adapters: one index for all tokens (the first adapter unless given), or
        integers of x's leading shape or of its first dimensions (one for each
        sequence of a batch); outside [0, L): none."""
        lead = x.shape[:-1]
        x2 = _tokens(x, self.in_features, "W8A8AdaptedLinear")
        codes = isinstance(x2, Tokens)
        rows = x2.codes if codes else x2
        if not isinstance(adapters, torch.Tensor):
            index = min(max(int(adapters), -1), self.a.shape[0])
            ids = torch.full((rows.shape[0],), index, dtype=torch.int32, device=rows.device)
        else:
            if adapters.dtype.is_floating_point or adapters.dtype in (torch.bool, torch.complex64, torch.complex128):
                raise TypeError(f"adapters must be integers (got {adapters.dtype})")
            if tuple(adapters.shape) != tuple(lead[:adapters.dim()]):
                raise ValueError(f"adapters of shape {tuple(adapters.shape)} are not those of tokens {tuple(lead)}")
            ids = adapters.reshape(*adapters.shape, *(1,) * (len(lead) - adapters.dim())).expand(lead)
            if ids.dtype != torch.int32:    # (what does not fit 32 bits is outside the set)
                ids = ids.to(torch.int64).clamp(-1, self.a.shape[0])
            ids = ids.reshape(-1).to(torch.int32).contiguous()
        args = (self.wq, self.w_scale)
        low = (self.a, self.b, ids, self.scaling)
        of_x = x2.stand_in is not None if codes else x2.requires_grad
        if torch.is_grad_enabled() and (of_x or self.a.requires_grad or self.b.requires_grad):
            x_in, xq, x_scale = (x2.stand_in, x2.codes, x2.scale) if codes else (x2, None, None)
            y = autograd._Adapted.apply(x_in, xq, x_scale, *args, self.bias, *low)
        elif codes:
            y = adapter_ops.linear_adapters(x2.codes, x2.scale, *args, *low, bias=self.bias)
        else:
            y = adapter_ops.linear_adapters_dynamic(x2, *args, *low, bias=self.bias)
        return y.reshape(*lead, self.out_features)


class W8A8RMSNorm(torch.nn.Module):
    """The residual's addition and the root-mean-square norm in front of W8A8
    modules, which take its codes: norm(x, residual) -> (Tokens, x + residual)."""

    def __init__(self, weight: torch.Tensor | None, eps: float = 1e-6):
        super().__init__()
        self.eps = eps
        self.register_parameter("weight", None if weight is None else
                                torch.nn.Parameter(weight.detach().to(torch.bfloat16).contiguous()))

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> tuple[Tokens, torch.Tensor]:
        K = x.shape[-1]
        if residual is not None and residual.shape != x.shape:
            raise ValueError("residual must have x's shape")
        x2 = _tokens(x, K, "W8A8RMSNorm")
        r2 = None if residual is None else _tokens(residual, K, "W8A8RMSNorm")
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x2, r2, self.weight)):
            xq, scale, stand_in, h = autograd._NormCodes.apply(x2, r2, self.weight, self.eps)
            stand_in = stand_in.reshape(x.shape)
        else:
            xq, scale, h = adapter_ops.add_rms_norm_quantize(x2, r2, self.weight, self.eps)
            stand_in = None
        return Tokens(xq.reshape(x.shape), scale.reshape(x.shape[:-1]), stand_in), h.reshape(x.shape)


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

    def forward(self, x: torch.Tensor | Tokens, adapters: torch.Tensor | int | None = None) -> torch.Tensor:
        """adapters: those of a W8A8AdaptedLinear as the down projection; without
        them its own default, the first adapter for every token."""
        x2 = _tokens(x, self.in_features, "W8A8GatedMLP")
        if isinstance(x2, Tokens):
            args = (self.wq, self.w_scale, self.bias)
            if x2.stand_in is not None:
                h = autograd._Gated.apply(x2.stand_in, *args, self.act, x2.codes, x2.scale)
            else:
                h = block_ops.gated_linear(x2.codes, x2.scale, *args, act=self.act)
        elif x2.requires_grad and torch.is_grad_enabled():
            h = autograd._Gated.apply(x2, self.wq, self.w_scale, self.bias, self.act)
        else:
            h = block_ops.gated_linear_dynamic(x2, self.wq, self.w_scale, self.bias, act=self.act)
        lead = x.shape[:-1]
        if adapters is not None:
            return self.down(h.reshape(*lead, self.down.in_features), adapters)
        return self.down(h).reshape(*lead, self.down.out_features)


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

    def forward(self, x: torch.Tensor | Tokens, cos: torch.Tensor, sin: torch.Tensor,
                positions: torch.Tensor | None = None, adapters: torch.Tensor | int | None = None):
        """x [..., features] -> q [..., Hq, D], k and v [..., Hk, D]; cos, sin
        fp32 [P, rot/2], positions int32, one per token.  Without positions a
        token is at its index in its sequence (the last dimension before the
        features), in sequences longer than the tables at that index mod P.
        adapters: those of a W8A8AdaptedLinear as the projection; without them its
        own default, the first adapter for every token."""
        if positions is None and x.dim() > 2:
            cos, sin = self._tables(x.shape[-2], x.shape[:-2].numel(), cos, sin)
        qkv = self.proj(x) if adapters is None else self.proj(x, adapters)
        qkv = qkv.reshape(-1, self.proj.out_features)
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
