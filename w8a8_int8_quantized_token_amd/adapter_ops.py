"""Binding of the norm that leaves codes and of the linear with low-rank
adapters: checks, output allocation and the call, as in ``block_ops``."""
from __future__ import annotations

import torch

from ._lib import lib, load_calls
from .block_ops import _call, _empty, _matrix, _on, _out, _ptr, _rows, _workspace

_calls = load_calls()
BF = torch.bfloat16


def add_rms_norm_quantize(x, residual=None, weight=None, eps: float = 1e-6, fp8: bool = False, h=None):
    """The residual's addition, the root-mean-square norm of each row and its
    codes: (xq int8 [M,K] or, ``fp8``, uint8 e4m3 bits; x_scale fp32 [M]; h =
    bf16(x + residual)).  x, residual bf16 [M,K], weight bf16 [K] or None.
    xq * x_scale is the normed row on the codes' grid (127 or 448 steps of the
    row's largest magnitude).  A row with a NaN or an infinity has a scale that
    is not finite.
    Without a residual h is x itself; a given h (it may be x or residual)
    receives the sum."""
    if h is None:
        out = _calls.add_rms_norm_quantize(x, residual, weight, eps, fp8)
        if out is not None:
            return out
    px, M, K, dev = _matrix(x, BF, "x")
    pr = None if residual is None else _on(residual, BF, (M, K), "residual", dev)
    pw = None if weight is None else _on(weight, BF, (K,), "weight", dev)
    if h is not None:
        ph = _on(h, BF, (M, K), "h", dev)
    elif residual is None:
        h, ph = x, None
    else:
        h = _empty((M, K), BF, dev)
        ph = h.data_ptr()
    xq = _empty((M, K), torch.uint8 if fp8 else torch.int8, dev)
    x_scale = _empty((M,), torch.float32, dev)
    _call(dev, lib.w8a8_add_rms_norm_quantize, px, pr, pw, ph, xq.data_ptr(), x_scale.data_ptr(), M, K, eps,
          int(bool(fp8)))
    return xq, x_scale, h


def add_rms_norm_backward(dn, h, weight=None, eps: float = 1e-6, dh=None, dweight: bool = True, dx=None,
                          workspace=None):
    """Gradients of ``add_rms_norm_quantize`` for dn (of the normed rows, bf16
    [M,K]) and dh (of h, from what else reads it; or None), the rounding to codes
    passed straight through: (dx bf16 [M,K], of x and of residual, new unless
    given: it may be dn, dh or h; fp32 gradient of the weight [K], None without
    ``dweight``)."""
    if dx is None and workspace is None:
        grads = _calls.add_rms_norm_backward(dn, h, weight, eps, dh, dweight)
        if grads is not None:
            return grads
    ph, M, K, dev = _matrix(h, BF, "h")
    pdn = _on(dn, BF, (M, K), "dn", dev)
    pdh = None if dh is None else _on(dh, BF, (M, K), "dh", dev)
    pw = None if weight is None else _on(weight, BF, (K,), "weight", dev)
    if dx is None:
        dx = _empty((M, K), BF, dev)
        pdx = dx.data_ptr()
    else:
        pdx = _on(dx, BF, (M, K), "dx", dev)
    gw = _empty((K,), torch.float32, dev) if dweight else None
    need = lib.w8a8_add_rms_norm_backward_workspace(M, K) if dweight else 0
    pws, nws, workspace = _workspace(workspace, need, dev)
    _call(dev, lib.w8a8_add_rms_norm_backward, pdn, pdh, ph, pw, pdx, _ptr(gw), M, K, eps, pws, nws)
    return dx, gw


def _adapters(a, b, ids, scaling, M, N, K, dev):
    """Addresses of a, b, scaling, ids, and the rank and number of adapters."""
    if not isinstance(a, torch.Tensor):
        raise TypeError("a must be a torch.Tensor")
    if a.dim() != 3:
        raise ValueError(f"a must be [adapters, rank, K] (got shape {tuple(a.shape)})")
    L, R = a.shape[:2]
    return (_on(a, BF, (L, R, K), "a", dev), _on(b, BF, (L, N, R), "b", dev),
            _on(scaling, torch.float32, (L,), "scaling", dev), _on(ids, torch.int32, (M,), "ids", dev)), R, L


def linear_adapters(xq, x_scale, wq, w_scale, a, b, ids, scaling, bias=None, y=None, tile: int = -1, workspace=None):
    """``linear`` with a low-rank adapter for each token: bf16 y [M,N] with
    sum_r t[m,r] b[ids[m]][n,r] added before the rounding, t = scaling[ids[m]] *
    x a[ids[m]]^T, x = xq * x_scale.  a bf16 [L,R,K], b bf16 [L,N,R], ids int32
    [M] (outside [0, L): no adapter), scaling fp32 [L]; R a multiple of 8 up to
    128."""
    if y is None and workspace is None and tile < 0 and x_scale is not None:
        out = _calls.linear_adapters(xq, x_scale, wq, w_scale, bias, a, b, ids, scaling)
        if out is not None:
            return out
    px, M, K, dev = _matrix(xq, torch.int8, "xq")
    N = _rows(wq, "wq")[0]
    pw = _on(wq, torch.int8, (N, K), "wq", dev)
    pxs = _on(x_scale, torch.float32, (M,), "x_scale", dev)
    ps = _on(w_scale, torch.float32, (N,), "w_scale", dev)
    pb = None if bias is None else _on(bias, BF, (N,), "bias", dev)
    low, R, L = _adapters(a, b, ids, scaling, M, N, K, dev)
    y, py = _out(y, (M, N), dev)
    pws, nws, workspace = _workspace(workspace, lib.w8a8_linear_adapters_workspace(M, N, K, R, 0), dev)
    _call(dev, lib.w8a8_linear_adapters, px, pxs, pw, ps, pb, *low, py, M, N, K, R, L, tile, pws, nws)
    return y


def linear_adapters_dynamic(x, wq, w_scale, a, b, ids, scaling, bias=None, y=None, workspace=None):
    """bf16 x [M,K] -> bf16 y [M,N]: ``quantize_act`` and ``linear_adapters`` in
    one call, the same bits; one or two launches for a few tokens."""
    if y is None and workspace is None:
        out = _calls.linear_adapters(x, None, wq, w_scale, bias, a, b, ids, scaling)
        if out is not None:
            return out
    px, M, K, dev = _matrix(x, BF, "x")
    N = _rows(wq, "wq")[0]
    pw = _on(wq, torch.int8, (N, K), "wq", dev)
    ps = _on(w_scale, torch.float32, (N,), "w_scale", dev)
    pb = None if bias is None else _on(bias, BF, (N,), "bias", dev)
    low, R, L = _adapters(a, b, ids, scaling, M, N, K, dev)
    y, py = _out(y, (M, N), dev)
    pws, nws, workspace = _workspace(workspace, lib.w8a8_linear_adapters_workspace(M, N, K, R, 1), dev)
    _call(dev, lib.w8a8_linear_adapters_dynamic, px, pw, ps, pb, *low, py, M, N, K, R, L, pws, nws)
    return y


def linear_adapters_backward(dy, xq, x_scale, wq, w_scale, a, b, ids, scaling, dx: bool = True, da: bool = True,
                             db: bool = True, workspace=None):
    """Gradients of ``linear_adapters`` for dy bf16 [M,N] on frozen codes of the
    weight, the rounding of the activations passed straight through: (dx bf16
    [M,K], da bf16 [L,R,K], db bf16 [L,N,R]), None where not asked for.  xq and
    x_scale may be None without da and db."""
    if workspace is None:
        grads = _calls.linear_adapters_backward(dy, xq, x_scale, wq, w_scale, a, b, ids, scaling, dx, da, db)
        if grads is not None:
            return grads
    pdy, M, N, dev = _matrix(dy, BF, "dy")
    K = _rows(wq, "wq")[1]
    pw = _on(wq, torch.int8, (N, K), "wq", dev)
    ps = _on(w_scale, torch.float32, (N,), "w_scale", dev)
    if xq is None and x_scale is None and not da and not db:
        pxq = pxs = None
    else:
        pxq = _on(xq, torch.int8, (M, K), "xq", dev)
        pxs = _on(x_scale, torch.float32, (M,), "x_scale", dev)
    low, R, L = _adapters(a, b, ids, scaling, M, N, K, dev)
    gx = _empty((M, K), BF, dev) if dx else None
    ga = _empty((L, R, K), BF, dev) if da else None
    gb = _empty((L, N, R), BF, dev) if db else None
    need = lib.w8a8_linear_adapters_backward_workspace(M, N, K, R, L, bool(dx), bool(da), bool(db))
    pws, nws, workspace = _workspace(workspace, need, dev)
    _call(dev, lib.w8a8_linear_adapters_backward, pdy, pxq, pxs, pw, ps, *low, _ptr(gx), _ptr(ga), _ptr(gb), M, N, K, R,
          L, pws, nws)
    return gx, ga, gb
