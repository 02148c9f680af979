"""Plain 64-bit forms of the norm that leaves codes and of the linear with
low-rank adapters (torch on the CPU), written from their formulas, and the
bounds of the errors that their kernels may make."""
from __future__ import annotations

import torch

import block_ref as ref

F64, BF = torch.float64, torch.bfloat16
U = 2.0 ** -24                       # half a step of fp32, relative
HALF = ref.BF16_HALF_STEP            # of bf16


def norm_codes(x, residual, w, eps, fp8):
    """(codes as values, scale in 64 bits, h): codes by the definition, whose
    fp32 scale and quotient belong to it."""
    h = x if residual is None else (x.float() + residual.float()).to(BF)
    v = h.float() if w is None else h.float() * w.float()
    top = 448.0 if fp8 else 127.0
    s = v.abs().amax(1) * (torch.tensor(1.0) / torch.tensor(top))
    q = (v / torch.where(s > 0, s, torch.ones_like(s))[:, None]).clamp(-top, top)
    q = q.to(torch.float8_e4m3fn).float() if fp8 else torch.round(q)
    q = torch.where(s[:, None] > 0, q, torch.zeros_like(q))
    rms = torch.sqrt(h.to(F64).square().mean(1) + eps)
    return q, torch.where(s > 0, s.to(F64) / rms, torch.zeros_like(rms)), h


def norm_grad(dn, dh, h, w, eps):
    """(dx, the terms' magnitudes that its fp32 errors scale with, dweight, its
    terms' magnitudes)."""
    dn, h = dn.to(F64), h.to(F64)
    w = torch.ones(h.shape[1], dtype=F64) if w is None else w.to(F64)
    power = h.square().mean(1, keepdim=True) + eps
    r = torch.where(power > 0, power.rsqrt(), torch.zeros_like(power))
    hh, d = h * r, dn * w
    dx = r * (d - hh * (d * hh).mean(1, keepdim=True))
    size = r * (d.abs() + hh.abs() * (d * hh).abs().mean(1, keepdim=True))
    if dh is not None:
        dx, size = dx + dh.to(F64), size + dh.to(F64).abs()
    return dx, size, (dn * hh).sum(0), (dn * hh).abs().sum(0)


def low(x, p, ids, scaling, transposed=False):
    """x [M,C] by each row's own p[id] [R,C] (or [C,R]), times its scaling, and
    the same of magnitudes; zeros for rows without one."""
    R = p.shape[2 if transposed else 1]
    t, size = x.new_zeros(x.shape[0], R), x.new_zeros(x.shape[0], R)
    for i in range(p.shape[0]):
        at = (ids == i).nonzero().flatten()
        q = p[i].to(F64) if transposed else p[i].to(F64).T
        s = scaling[i].to(F64)
        t[at], size[at] = s * (x[at] @ q), s.abs() * (x[at].abs() @ q.abs())
    return t, size


def up(t, p, ids, transposed=False):
    """t [M,R] by each row's own p[id] [C,R] (or [R,C])."""
    y = t.new_zeros(t.shape[0], p.shape[2 if transposed else 1])
    for i in range(p.shape[0]):
        at = (ids == i).nonzero().flatten()
        y[at] = t[at] @ (p[i].to(F64) if transposed else p[i].to(F64).T)
    return y


def linear(xq, xs, wq, ws, a, b, ids, scaling, bias):
    """(y, the bound of its errors before the last rounding): t's rounding to
    bf16 is half a step of each of its terms; fp32 sums of n terms are off by at
    most n units of their terms' magnitudes (in any order; twice that for the
    matrix cores' own additions); the linear's own few roundings."""
    K, R = xq.shape[1], a.shape[1]
    x = xq.to(F64) * xs.to(F64)[:, None]
    p = ref.product(xq, xs, wq, ws, None)
    t, t_size = low(x, a, ids, scaling)
    y = p + up(t, b, ids)
    bound = 8 * U * (p.abs() + (0 if bias is None else bias.to(F64).abs()))
    slack = up(t.abs() * HALF + t_size * (2 * K * U) + t.abs() * (2 * R + 8) * U, b.abs(), ids)
    return (y if bias is None else y + bias.to(F64)), bound + slack


def grads(dy, xq, xs, wq, ws, a, b, ids, scaling):
    """((dx, bound), (da, bound), (db, bound)): the products' operands that are
    rounded to bf16 once are half a step off each, and their fp32 sums as above."""
    M, N = dy.shape
    K, R = xq.shape[1], a.shape[1]
    x, dy = xq.to(F64) * xs.to(F64)[:, None], dy.to(F64)
    w = wq.to(F64) * ws.to(F64)[:, None]
    t, t_size = low(x, a, ids, scaling)
    u, u_size = low(dy, b, ids, scaling, transposed=True)
    t_off = t.abs() * HALF + t_size * (2 * K * U)
    u_off = u.abs() * HALF + u_size * (2 * N * U)
    dx = dy @ w + up(u, a, ids, transposed=True)
    dx_off = (dy.abs() @ w.abs()) * (HALF + 2 * N * U) + up(u_off + u.abs() * 2 * R * U, a.abs(), ids, transposed=True)
    da, da_off = x.new_zeros(a.shape), x.new_zeros(a.shape)
    db, db_off = x.new_zeros(b.shape), x.new_zeros(b.shape)
    for i in range(a.shape[0]):
        at = (ids == i).nonzero().flatten()
        n = len(at)
        da[i], da_off[i] = u[at].T @ x[at], (u_off[at] + u[at].abs() * (2 * n + 4) * U).T @ x[at].abs()
        db[i], db_off[i] = dy[at].T @ t[at], dy[at].abs().T @ (t_off[at] + t[at].abs() * (2 * n + 4) * U)
    return (dx, dx_off), (da, da_off), (db, db_off)
