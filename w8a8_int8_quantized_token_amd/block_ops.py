"""Binding of the operators around the linear: the few-token forms from bf16
activations, the gated product, the backward passes, and the norm and rotation
of queries and keys.

As in ``ops``: argument checks, output allocation with torch and the call on
the current stream of the tensors' device.  Tensors of one call are on one
device (it need not be the current one).  Workspaces are allocated per call
from torch's caching allocator, on the call's stream, unless given.
"""
from __future__ import annotations

import torch

from ._lib import check, lib

ACTS = {"silu": 0, "gelu": 1}


def _on(t, dtype, shape, name, device=None):
    """t's address, checked: a contiguous device tensor of that type and shape
    (None in a shape: any size), on `device` where given."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    got = t.shape
    if len(got) != len(shape) or any(w is not None and w != g for w, g in zip(shape, got)):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(got)})")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, other tensors on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _call(device, fn, *args):
    """fn(*args, stream) with the tensors' device current."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            status = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    else:
        status = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    check(status, fn.__name__)


def _workspace(given, need, device):
    """(address, bytes) of the call's workspace and the tensor that holds it."""
    if given is None:
        if need == 0:
            return None, 0, None
        given = torch.empty((need,), dtype=torch.uint8, device=device)
    return _on(given, torch.uint8, (None,), "workspace", device), given.numel(), given


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)} (got {act!r})")
    return ACTS[act]


def _dynamic(fn, workspace_fn, x, wq, w_scale, bias, y, per, act, workspace):
    px = _on(x, torch.bfloat16, (None, None), "x")
    M, K = x.shape
    dev = x.device
    pw = _on(wq, torch.int8, (None, K), "wq", dev)
    rows = wq.shape[0]
    if rows % per:
        raise ValueError("wq must hold as many gate rows as up rows")
    N = rows // per
    ps = _on(w_scale, torch.float32, (rows,), "w_scale", dev)
    pb = None if bias is None else _on(bias, torch.bfloat16, (rows,), "bias", dev)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    py = _on(y, torch.bfloat16, (M, N), "y", dev)
    pws, nws, workspace = _workspace(workspace, workspace_fn(M, N, K), dev)
    _call(dev, fn, px, pw, ps, pb, py, M, N, K, act, pws, nws)
    return y


def linear_dynamic(x, wq, w_scale, bias=None, y=None, gelu: bool = False, workspace=None):
    """bf16 x [M,K] -> bf16 y [M,N]: ``quantize_act`` and ``linear`` in one
    call, the same bits; one launch for a few tokens."""
    return _dynamic(lib.w8a8_linear_dynamic, lib.w8a8_linear_dynamic_workspace, x, wq, w_scale, bias, y, 1,
                    int(bool(gelu)), workspace)


def gated_linear_dynamic(x, wq, w_scale, bias=None, y=None, act: str = "silu", workspace=None):
    """bf16 x [M,K] -> bf16 y [M,N]: ``quantize_act`` and ``gated_linear`` in
    one call, the same bits; one launch for a few tokens."""
    return _dynamic(lib.w8a8_gated_linear_dynamic, lib.w8a8_gated_linear_dynamic_workspace, x, wq, w_scale, bias,
                    y, 2, _act(act), workspace)


def gated_linear(xq, x_scale, wq, w_scale, bias=None, y=None, act: str = "silu", tile: int = -1):
    """Gated product: bf16 y [M,N] = act(gate) * up, gate and up being
    ``linear``'s values for the first and the last N rows of wq [2N,K]."""
    a = _act(act)
    px = _on(xq, torch.int8, (None, None), "xq")
    M, K = xq.shape
    dev = xq.device
    pw = _on(wq, torch.int8, (None, K), "wq", dev)
    rows = wq.shape[0]
    if rows % 2:
        raise ValueError("wq must hold as many gate rows as up rows")
    pxs = _on(x_scale, torch.float32, (M,), "x_scale", dev)
    ps = _on(w_scale, torch.float32, (rows,), "w_scale", dev)
    pb = None if bias is None else _on(bias, torch.bfloat16, (rows,), "bias", dev)
    if y is None:
        y = torch.empty((M, rows // 2), dtype=torch.bfloat16, device=dev)
    py = _on(y, torch.bfloat16, (M, rows // 2), "y", dev)
    _call(dev, lib.w8a8_gated_linear_tile, px, pxs, pw, ps, pb, py, M, rows // 2, K, a, tile)
    return y


def _grads(dev, M, rows, K, dx, dw, dbias):
    bf = torch.bfloat16
    return (torch.empty((M, K), dtype=bf, device=dev) if dx else None,
            torch.empty((rows, K), dtype=bf, device=dev) if dw else None,
            torch.empty((rows,), dtype=bf, device=dev) if dbias else None)


def _ptr(t):
    return None if t is None else t.data_ptr()


def linear_backward(dy, xq, x_scale, wq, w_scale, dx: bool = True, dw: bool = True, dbias: bool = True,
                    workspace=None):
    """Gradients of ``linear`` (without GELU) for dy bf16 [M,N], the rounding
    to codes passed straight through: (dx bf16 [M,K], dw bf16 [N,K], dbias bf16
    [N]), None where not asked for.  xq and x_scale may be None without dw."""
    pdy = _on(dy, torch.bfloat16, (None, None), "dy")
    M, N = dy.shape
    dev = dy.device
    pw = _on(wq, torch.int8, (N, None), "wq", dev)
    K = wq.shape[1]
    ps = _on(w_scale, torch.float32, (N,), "w_scale", dev)
    if xq is None and x_scale is None and not dw:
        pxq = pxs = None
    else:
        pxq = _on(xq, torch.int8, (M, K), "xq", dev)
        pxs = _on(x_scale, torch.float32, (M,), "x_scale", dev)
    gx, gw, gb = _grads(dev, M, N, K, dx, dw, dbias)
    need = lib.w8a8_linear_backward_workspace(M, N, K, bool(dx), bool(dw), bool(dbias))
    pws, nws, workspace = _workspace(workspace, need, dev)
    _call(dev, lib.w8a8_linear_backward, pdy, pxq, pxs, pw, ps, _ptr(gx), _ptr(gw), _ptr(gb), M, N, K, pws, nws)
    return gx, gw, gb


def gated_linear_backward(dy, xq, x_scale, wq, w_scale, bias=None, act: str = "silu", dx: bool = True,
                          dw: bool = True, dbias: bool = True, workspace=None):
    """Gradients of ``gated_linear`` for dy bf16 [M,N], the rounding to codes
    passed straight through: (dx bf16 [M,K], dw bf16 [2N,K], dbias bf16 [2N]),
    None where not asked for."""
    a = _act(act)
    pdy = _on(dy, torch.bfloat16, (None, None), "dy")
    M, N = dy.shape
    dev = dy.device
    pw = _on(wq, torch.int8, (2 * N, None), "wq", dev)
    K = wq.shape[1]
    pxq = _on(xq, torch.int8, (M, K), "xq", dev)
    pxs = _on(x_scale, torch.float32, (M,), "x_scale", dev)
    ps = _on(w_scale, torch.float32, (2 * N,), "w_scale", dev)
    pb = None if bias is None else _on(bias, torch.bfloat16, (2 * N,), "bias", dev)
    gx, gw, gb = _grads(dev, M, 2 * N, K, dx, dw, dbias)
    need = lib.w8a8_gated_linear_backward_workspace(M, N, K, bool(dx), bool(dw), bool(dbias))
    pws, nws, workspace = _workspace(workspace, need, dev)
    _call(dev, lib.w8a8_gated_linear_backward, pdy, pxq, pxs, pw, ps, pb, _ptr(gx), _ptr(gw), _ptr(gb), M, N, K, a,
          pws, nws)
    return gx, gw, gb


def _heads(t, name, M=None, D=None, device=None, heads=None):
    """(address, row stride, head stride) of bf16 [M, heads, D], last dimension dense."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bf16 (got {t.dtype})")
    s = t.shape
    if len(s) != 3 or (M is not None and (s[0] != M or s[2] != D)) or (heads is not None and s[1] != heads):
        raise ValueError(f"{name} must be [rows, heads, head size] like its partners (got {tuple(s)})")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on the device of the other tensors (got {t.device})")
    row, head, last = t.stride()
    if last != 1 and s[2] > 1:
        raise ValueError(f"{name} must be dense along the head")
    # the stride of a dimension of one element is never used
    return t.data_ptr(), row if s[0] > 1 else 0, head if s[1] > 1 else 0


def _out_heads(t, name, like, D, device):
    """An output's view: no two of its elements may share an address."""
    v = _heads(t, name, like.shape[0], D, device, like.shape[1])
    (M, H, _), (row, head) = t.shape, v[1:]
    if H > 1 and abs(head) < D or M > 1 and abs(row) < D or \
            (M > 1 and H > 1 and not (abs(row) >= (H - 1) * abs(head) + D or abs(head) >= (M - 1) * abs(row) + D)):
        raise ValueError(f"{name} must not overlap itself")
    return v


def _rope_args(q, k, q_weight, k_weight, cos, sin, positions):
    vq = _heads(q, "q")
    M, Hq, D = q.shape
    dev = q.device
    vk = _heads(k, "k", M, D, dev)
    pqw = None if q_weight is None else _on(q_weight, torch.bfloat16, (D,), "q_weight", dev)
    pkw = None if k_weight is None else _on(k_weight, torch.bfloat16, (D,), "k_weight", dev)
    pc = _on(cos, torch.float32, (None, None), "cos", dev)
    P, half = cos.shape
    ps = _on(sin, torch.float32, (P, half), "sin", dev)
    pp = None if positions is None else _on(positions, torch.int32, (M,), "positions", dev)
    return vq, vk, (pqw, pkw, pc, ps, pp), (M, P, Hq, k.shape[1], D, 2 * half), dev


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None):
    """RMS norm of each head of q [M,Hq,D] and k [M,Hk,D] (bf16, any row and
    head strides, so views of a packed QKV matrix) and the rotation of their
    first 2 * cos.shape[1] values by cos, sin fp32 [P, rot/2] at each row's
    position (int32 [M]; None: row mod P).  q_weight, k_weight: bf16 [D] or
    None.  Returns (q_out, k_out), new dense tensors unless given; they may be
    q and k themselves.  Rows at a position outside [0, P) become zeros."""
    vq, vk, ptrs, sizes, dev = _rope_args(q, k, q_weight, k_weight, cos, sin, positions)
    D = sizes[4]
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
    if k_out is None:
        k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=dev)
    vqo, vko = _out_heads(q_out, "q_out", q, D, dev), _out_heads(k_out, "k_out", k, D, dev)
    _call(dev, lib.w8a8_qk_norm_rope, *vq, *vk, *ptrs, *vqo, *vko, *sizes, eps, int(bool(interleaved)))
    return q_out, k_out


def qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, cos, sin, positions=None, eps: float = 1e-6,
                          interleaved: bool = False, weights: bool = True, workspace=None):
    """Gradients of ``qk_norm_rope`` for the outputs' gradients dq [M,Hq,D],
    dk [M,Hk,D] (bf16, any row and head strides): (gradient of q, of k,
    bf16; of q_weight, of k_weight, fp32 [D], None without ``weights``)."""
    vq, vk, ptrs, sizes, dev = _rope_args(q, k, q_weight, k_weight, cos, sin, positions)
    M, _, Hq, Hk, D, _ = sizes
    vdq, vdk = _heads(dq, "dq", M, D, dev, Hq), _heads(dk, "dk", M, D, dev, Hk)
    gq = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
    gk = torch.empty(k.shape, dtype=torch.bfloat16, device=dev)
    gqw = gkw = None
    need = 0
    if weights:
        gqw = torch.empty((D,), dtype=torch.float32, device=dev)
        gkw = torch.empty((D,), dtype=torch.float32, device=dev)
        need = lib.w8a8_qk_norm_rope_backward_workspace(M, Hq, Hk, D)
    pws, nws, workspace = _workspace(workspace, need, dev)
    _call(dev, lib.w8a8_qk_norm_rope_backward, *vdq, *vdk, *vq, *vk, *ptrs, gq.data_ptr(), Hq * D, D, gk.data_ptr(),
          Hk * D, D, _ptr(gqw), _ptr(gkw), *sizes, eps, int(bool(interleaved)), pws, nws)
    return gq, gk, gqw, gkw
