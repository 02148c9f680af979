"""Binding of the operators around the linear: the few-token forms from bf16
activations, the gated product, the backward passes, and the norm and rotation
of queries and keys.

As in ``ops``: argument checks, output allocation with torch and the call on
the current stream of the tensors' device.  Tensors of one call are on one
device (it need not be the current one).  Workspaces are allocated per call
from torch's caching allocator, on the call's stream, unless given.

A plain call (no output or workspace given, every argument as it should be, the
tensors on the current device) is made in one native step by ``_calls``, which
gives None, with nothing launched, where it is not one; the code here then
makes the call or names what is wrong.
"""
from __future__ import annotations

import torch

from ._lib import check, lib, load_calls

_calls = load_calls()
ACTS = {"silu": 0, "gelu": 1}


def _on(t, dtype, shape, name, device):
    """t's address, checked: a contiguous tensor of that type and shape on
    the CUDA device of that index (one expression where all is well: these
    checks are most of a small call's host time)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device >= 0 and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, other tensors on device {device}")
    raise ValueError(f"{name} must be contiguous")


def _matrix(t, dtype, name):
    """(address, rows, columns, device index) of the matrix that the call's
    other tensors go by."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D (got shape {tuple(shape)})")
    device = t.get_device()
    return _on(t, dtype, shape, name, device), shape[0], shape[1], device


def _rows(t, name):
    """Rows and columns of a weight, whose type and place are checked later."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D (got shape {tuple(t.shape)})")
    return t.shape


def _call(device, fn, *args):
    """fn(*args, stream) with the tensors' device current."""
    stream = torch._C._cuda_getCurrentRawStream(device)   # current_stream(device).cuda_stream
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            status = fn(*args, stream)
    else:
        status = fn(*args, stream)
    if status:
        check(status, fn.__name__)


def _empty(shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=_DEVICES[device])


class _Devices(dict):
    """torch.device objects by index, made once."""

    def __missing__(self, index):
        self[index] = torch.device("cuda", index)
        return self[index]


_DEVICES = _Devices()


def _workspace(given, need, device):
    """(address, bytes, tensor that holds them) of the call's workspace."""
    if given is None:
        if need == 0:
            return None, 0, None
        given = _empty((need,), torch.uint8, device)
        return given.data_ptr(), need, given
    if not isinstance(given, torch.Tensor) or given.dim() != 1:
        raise ValueError("workspace must be a 1-D uint8 device tensor")
    return _on(given, torch.uint8, given.shape, "workspace", device), given.numel(), given


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)} (got {act!r})")
    return ACTS[act]


def _out(y, shape, device):
    """The given output's address, checked, or a new one."""
    if y is None:
        y = _empty(shape, torch.bfloat16, device)
        return y, y.data_ptr()
    return y, _on(y, torch.bfloat16, shape, "y", device)


def _dynamic(fn, workspace_fn, x, wq, w_scale, bias, y, per, act, workspace):
    px, M, K, dev = _matrix(x, torch.bfloat16, "x")
    rows = _rows(wq, "wq")[0]
    pw = _on(wq, torch.int8, (rows, K), "wq", dev)
    if rows % per:
        raise ValueError("wq must hold as many gate rows as up rows")
    N = rows // per
    ps = _on(w_scale, torch.float32, (rows,), "w_scale", dev)
    pb = None if bias is None else _on(bias, torch.bfloat16, (rows,), "bias", dev)
    y, py = _out(y, (M, N), dev)
    pws, nws, workspace = _workspace(workspace, workspace_fn(M, N, K), dev)
    _call(dev, fn, px, pw, ps, pb, py, M, N, K, act, pws, nws)
    return y


def linear_dynamic(x, wq, w_scale, bias=None, y=None, gelu: bool = False, workspace=None):
    """bf16 x [M,K] -> bf16 y [M,N]: ``quantize_act`` and ``linear`` in one
    call, the same bits; one launch for a few tokens."""
    if y is None and workspace is None:
        out = _calls.dynamic(x, wq, w_scale, bias, 1 if gelu else 0, 1)
        if out is not None:
            return out
    return _dynamic(lib.w8a8_linear_dynamic, lib.w8a8_linear_dynamic_workspace, x, wq, w_scale, bias, y, 1,
                    int(bool(gelu)), workspace)


def gated_linear_dynamic(x, wq, w_scale, bias=None, y=None, act: str = "silu", workspace=None):
    """bf16 x [M,K] -> bf16 y [M,N]: ``quantize_act`` and ``gated_linear`` in
    one call, the same bits; one launch for a few tokens."""
    if y is None and workspace is None:
        out = _calls.dynamic(x, wq, w_scale, bias, _act(act), 2)
        if out is not None:
            return out
    return _dynamic(lib.w8a8_gated_linear_dynamic, lib.w8a8_gated_linear_dynamic_workspace, x, wq, w_scale, bias,
                    y, 2, _act(act), workspace)


def gated_linear(xq, x_scale, wq, w_scale, bias=None, y=None, act: str = "silu", tile: int = -1):
    """Gated product: bf16 y [M,N] = act(gate) * up, gate and up being
    ``linear``'s values for the first and the last N rows of wq [2N,K]."""
    a = _act(act)
    px, M, K, dev = _matrix(xq, torch.int8, "xq")
    rows = _rows(wq, "wq")[0]
    pw = _on(wq, torch.int8, (rows, K), "wq", dev)
    if rows % 2:
        raise ValueError("wq must hold as many gate rows as up rows")
    pxs = _on(x_scale, torch.float32, (M,), "x_scale", dev)
    ps = _on(w_scale, torch.float32, (rows,), "w_scale", dev)
    pb = None if bias is None else _on(bias, torch.bfloat16, (rows,), "bias", dev)
    y, py = _out(y, (M, rows // 2), dev)
    _call(dev, lib.w8a8_gated_linear_tile, px, pxs, pw, ps, pb, py, M, rows // 2, K, a, tile)
    return y


def _grads(dev, M, rows, K, dx, dw, dbias):
    bf = torch.bfloat16
    return (_empty((M, K), bf, dev) if dx else None, _empty((rows, K), bf, dev) if dw else None,
            _empty((rows,), bf, dev) if dbias else None)


def _ptr(t):
    return None if t is None else t.data_ptr()


def linear_backward(dy, xq, x_scale, wq, w_scale, dx: bool = True, dw: bool = True, dbias: bool = True,
                    workspace=None):
    """Gradients of ``linear`` (without GELU) for dy bf16 [M,N], the rounding
    to codes passed straight through: (dx bf16 [M,K], dw bf16 [N,K], dbias bf16
    [N]), None where not asked for.  xq and x_scale may be None without dw."""
    if workspace is None:
        grads = _calls.backward(dy, xq, x_scale, wq, w_scale, None, -1, dx, dw, dbias)
        if grads is not None:
            return grads
    pdy, M, N, dev = _matrix(dy, torch.bfloat16, "dy")
    K = _rows(wq, "wq")[1]
    pw = _on(wq, torch.int8, (N, K), "wq", dev)
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
    if workspace is None:
        grads = _calls.backward(dy, xq, x_scale, wq, w_scale, bias, a, dx, dw, dbias)
        if grads is not None:
            return grads
    pdy, M, N, dev = _matrix(dy, torch.bfloat16, "dy")
    K = _rows(wq, "wq")[1]
    pw = _on(wq, torch.int8, (2 * N, K), "wq", dev)
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


def _heads(t, shape, name, device):
    """Address, row stride and head stride of bf16 [M, heads, D], dense along D."""
    try:
        row, head, last = t.stride()
        if t.dtype is torch.bfloat16 and t.shape == shape and t.get_device() == device >= 0 and last == 1:
            # the stride of a dimension of one element is never used
            return t.data_ptr(), row if shape[0] > 1 else 0, head if shape[1] > 1 else 0
    except (AttributeError, ValueError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bf16 (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{name} must be on the device of the other tensors (got {t.device})")
    raise ValueError(f"{name} must be dense along the head")


def _out_heads(t, shape, name, device):
    """An output and its view, new where not given; no two elements of a
    given one may share an address."""
    M, H, D = shape
    if t is None:
        t = _empty(shape, torch.bfloat16, device)
        return t, (t.data_ptr(), H * D, D)
    v = _heads(t, shape, name, device)
    row, head = v[1:]
    if (H > 1 and head < D) or (M > 1 and row < D) or \
            (M > 1 and H > 1 and row < (H - 1) * head + D and head < (M - 1) * row + D):
        raise ValueError(f"{name} must not overlap itself")
    return t, v


def _rope_args(q, k, q_weight, k_weight, cos, sin, positions):
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor):
        raise TypeError("q and k must be torch.Tensors")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [rows, heads, head size]")
    dev = q.get_device()
    M, Hq, D = q.shape
    Hk = k.shape[1]
    vq, vk = _heads(q, q.shape, "q", dev), _heads(k, (M, Hk, D), "k", dev)
    pqw = None if q_weight is None else _on(q_weight, torch.bfloat16, (D,), "q_weight", dev)
    pkw = None if k_weight is None else _on(k_weight, torch.bfloat16, (D,), "k_weight", dev)
    pc, P, half, _ = _matrix(cos, torch.float32, "cos")
    ps = _on(sin, torch.float32, (P, half), "sin", dev)
    if cos.get_device() != dev:
        raise ValueError(f"cos is on {cos.device}, other tensors on device {dev}")
    pp = None if positions is None else _on(positions, torch.int32, (M,), "positions", dev)
    return vq, vk, (pqw, pkw, pc, ps, pp), (M, P, Hq, Hk, D, 2 * half), dev


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None):
    """RMS norm of each head of q [M,Hq,D] and k [M,Hk,D] (bf16, any row and
    head strides, so views of a packed QKV matrix) and the rotation of their
    first 2 * cos.shape[1] values by cos, sin fp32 [P, rot/2] at each row's
    position (int32 [M]; None: row mod P).  q_weight, k_weight: bf16 [D] or
    None.  Returns (q_out, k_out), new dense tensors unless given; they may be
    q and k themselves and overlap nothing otherwise.  Rows at a position outside [0, P) become zeros, also
    where the tables have no columns (the norm alone)."""
    if q_out is None and k_out is None:
        out = _calls.qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)
        if out is not None:
            return out
    vq, vk, ptrs, sizes, dev = _rope_args(q, k, q_weight, k_weight, cos, sin, positions)
    q_out, vqo = _out_heads(q_out, q.shape, "q_out", dev)
    k_out, vko = _out_heads(k_out, k.shape, "k_out", dev)
    _call(dev, lib.w8a8_qk_norm_rope, *vq, *vk, *ptrs, *vqo, *vko, *sizes, eps, int(bool(interleaved)))
    return q_out, k_out


def qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, cos, sin, positions=None, eps: float = 1e-6,
                          interleaved: bool = False, weights: bool = True, workspace=None, q_grad=None, k_grad=None):
    """Gradients of ``qk_norm_rope`` for the outputs' gradients dq [M,Hq,D],
    dk [M,Hk,D] (bf16, any row and head strides): (gradient of q, of k,
    bf16, new tensors unless given as q_grad, k_grad; of q_weight, of k_weight,
    fp32 [D], None without ``weights``)."""
    if workspace is None and q_grad is None and k_grad is None:
        grads = _calls.qk_norm_rope_backward(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, dq, dk,
                                             weights)
        if grads is not None:
            return grads
    vq, vk, ptrs, sizes, dev = _rope_args(q, k, q_weight, k_weight, cos, sin, positions)
    M, _, Hq, Hk, D, _ = sizes
    vdq, vdk = _heads(dq, q.shape, "dq", dev), _heads(dk, k.shape, "dk", dev)
    gq, vgq = _out_heads(q_grad, q.shape, "q_grad", dev)
    gk, vgk = _out_heads(k_grad, k.shape, "k_grad", dev)
    gqw = gkw = None
    need = 0
    if weights:
        gqw, gkw = _empty((2, D), torch.float32, dev)
        need = lib.w8a8_qk_norm_rope_backward_workspace(M, Hq, Hk, D)
    pws, nws, workspace = _workspace(workspace, need, dev)
    _call(dev, lib.w8a8_qk_norm_rope_backward, *vdq, *vdk, *vq, *vk, *ptrs, *vgq, *vgk, _ptr(gqw),
          _ptr(gkw), *sizes, eps, int(bool(interleaved)), pws, nws)
    return gq, gk, gqw, gkw
