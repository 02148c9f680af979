"""Plain 64-bit forms of the operators around the linear (numpy-like torch on
the CPU), written from their formulas, and the error bounds the tests use."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
BF16_HALF_STEP = torch.finfo(torch.bfloat16).eps / 2    # 2^-8, relative


def codes_of(x):
    """bf16 [R,K] -> (codes, scales) by the definition: scale = fl32(amax / 127),
    code = rne(fl32(x / scale))."""
    x = x.float()
    s = x.abs().amax(1) / torch.tensor(127.0)
    q = torch.round(x / torch.where(s > 0, s, torch.ones_like(s))[:, None]).clamp(-127, 127)
    return q.to(torch.int8), s


def phi(v):
    return 0.5 * (1.0 + torch.erf(v / math.sqrt(2.0)))


def act(v, kind):
    return v * torch.sigmoid(v) if kind == "silu" else v * phi(v)


def act_slope(v, kind):
    if kind == "silu":
        s = torch.sigmoid(v)
        return s * (1 + v * (1 - s))
    return phi(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)


def product(xq, xs, wq, ws, bias):
    y = (xq.to(F64) @ wq.to(F64).T) * xs.to(F64)[:, None] * ws.to(F64)
    return y if bias is None else y + bias.to(F64)


def gated(xq, xs, wq, ws, bias, kind):
    g, u = product(xq, xs, wq, ws, bias).chunk(2, 1)
    return act(g, kind) * u


def product_grads(d, xq, xs, wq, ws):
    """(dx, dw, dbias) of the product for d [M, rows], with the sums of the
    terms' magnitudes that bound their rounding."""
    w, x = wq.to(F64) * ws.to(F64)[:, None], xq.to(F64) * xs.to(F64)[:, None]
    return ((d @ w, d.abs() @ w.abs()), (d.T @ x, d.abs().T @ x.abs()), (d.sum(0), d.abs().sum(0)))


def gated_d(dy, xq, xs, wq, ws, bias, kind):
    g, u = product(xq, xs, wq, ws, bias).chunk(2, 1)
    dy = dy.to(F64)
    return torch.cat([dy * u * act_slope(g, kind), dy * act(g, kind)], 1)


def turned(n, cos, sin, rot, interleaved, back=False):
    """n [M,H,D] with the pairs of its first rot values turned; cos, sin [M, rot/2]."""
    c, s = cos.to(F64)[:, None], sin.to(F64)[:, None] * (-1 if back else 1)
    out = n.clone()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    a, b = n[..., ia], n[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    return out


def norm_rope(x, w, cos, sin, eps, interleaved):
    x = x.to(F64)
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        n = n * w.to(F64)
    return turned(n, cos, sin, 2 * cos.shape[1], interleaved)


def norm_rope_grad(dy, x, w, cos, sin, eps, interleaved):
    x = x.to(F64)
    w = torch.ones(x.shape[-1], dtype=F64) if w is None else w.to(F64)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    dn = turned(dy.to(F64), cos, sin, 2 * cos.shape[1], interleaved, back=True)
    xh = x * r
    dx = r * (dn * w - xh * (dn * w * xh).mean(-1, keepdim=True))
    return dx, (dn * xh).sum((0, 1)), (dn * xh).abs().sum((0, 1))


def rms(v):
    return float(v.to(F64).square().mean().sqrt()) if v.numel() else 0.0


def check(got, ref, slack, what, rms_steps=1.0):
    """|got - ref| <= half a bf16 step of ref + slack (an elementwise bound of
    the other errors), and the error's rms within `rms_steps` half steps."""
    got, ref = got.detach().cpu().to(F64), ref.cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), what
    err = (got - ref).abs()
    # the rounded value's step is at most that of |ref| + slack
    bound = BF16_HALF_STEP * (ref.abs() + slack) + slack
    over = (err - bound).max() if err.numel() else torch.tensor(0.0)
    assert float(over) <= 0, (what, float(over), float(err.max()))
    assert rms(err) <= rms_steps * BF16_HALF_STEP * rms(ref) + 1e-30, (what, rms(err), rms(ref))


def norm_rope_any(x, w, cos, sin, eps):
    """norm_rope with halves paired, written with differentiable operations."""
    rot = 2 * cos.shape[1]
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(F64)
    c, s = cos.to(F64)[:, None], sin.to(F64)[:, None]
    a, b = n[..., :rot // 2], n[..., rot // 2:rot]
    return torch.cat([a * c - b * s, b * c + a * s, n[..., rot:]], -1)
