"""Host-side checks of the operators around the linear: refusals before any
launch (fake pointers, never dereferenced), the binding's argument checks, and
the gradients' formulas against differences."""
import ctypes

import pytest
import torch

import block_ref as ref

A = 0x10000
BF = torch.bfloat16


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_quantized_token_amd as pkg
    return pkg


NULL, SHAPE, ALIGN, ARG = 1, 2, 3, 5


@pytest.mark.parametrize("name,per", [("linear", 1), ("gated_linear", 2)])
def test_dynamic_refusals(w8, name, per):
    f = getattr(w8.lib, f"w8a8_{name}_dynamic")
    ws = getattr(w8.lib, f"w8a8_{name}_dynamic_workspace")

    def call(x=A, wq=A, sw=A, b=A, y=A, M=4, N=8, K=64, act=0, w=None, n=0):
        return f(x, wq, sw, b, y, M, N, K, act, w, n, None)

    for M, N, K in [(-1, 8, 64), (4, 0, 64), (4, 8, 0), (4, 8, 24), (4, 8, 133152), (2 ** 26 + 1, 8, 64),
                    (4, 2 ** 26 // per + 1, 64)]:
        assert call(M=M, N=N, K=K) == SHAPE, (M, N, K)
        assert ws(M, N, K) == 0
    assert call(M=0, x=None, y=None) == 0
    for k in ("x", "wq", "sw", "y"):
        assert call(**{k: None}) == NULL
    assert call(x=A + 2) == ALIGN and call(wq=A + 8) == ALIGN and call(sw=A + 2) == ALIGN
    assert call(y=A + 1) == ALIGN and call(b=A + 1) == ALIGN
    assert ws(4, 8, 64) == 0 and ws(16, 8, 64) == 0 and ws(1, 8, 16384) == 0
    assert ws(17, 8, 64) >= 17 * 64 + 17 * 4                    # more tokens: codes in the workspace
    need = ws(33, 8, 64)
    assert need >= 33 * 64 + 33 * 4
    assert call(M=33) == NULL                                   # a workspace is needed
    assert call(M=33, w=A, n=need - 1) == ARG
    assert call(M=33, w=A + 4, n=need) == ALIGN
    if per == 2:
        assert call(act=2) == ARG and call(act=-1) == ARG
    # codes that do not fit a compute unit's LDS are made in the workspace
    assert ws(2, 8, 16384) >= 2 * 16384


def test_gated_refusals(w8):
    def call(xq=A, xs=A, wq=A, sw=A, b=A, y=A, M=4, N=8, K=64, act=0, tile=-1):
        return w8.lib.w8a8_gated_linear_tile(xq, xs, wq, sw, b, y, M, N, K, act, tile, None)

    for M, N, K in [(-1, 8, 64), (4, 0, 64), (4, 8, 8), (4, 8, 72), (4, 8, 133152), (4, 2 ** 25 + 1, 64)]:
        assert call(M=M, N=N, K=K) == SHAPE
    assert call(act=2) == ARG and call(act=-1) == ARG and call(tile=w8.num_tiles()) == ARG
    assert call(M=0, xq=None) == 0
    for k in ("xq", "xs", "wq", "sw", "y"):
        assert call(**{k: None}) == NULL
    assert call(xq=A + 4) == ALIGN and call(wq=A + 1) == ALIGN and call(xs=A + 2) == ALIGN
    assert call(y=A + 1) == ALIGN and call(b=A + 1) == ALIGN and call(sw=A + 1) == ALIGN


@pytest.mark.parametrize("gated", [False, True])
def test_backward_refusals(w8, gated):
    name = "w8a8_gated_linear_backward" if gated else "w8a8_linear_backward"
    f, wsf = getattr(w8.lib, name), getattr(w8.lib, name + "_workspace")

    def call(dy=A, xq=A, xs=A, wq=A, sw=A, b=A, dx=A, dw=A, db=A, M=4, N=8, K=64, act=0, w=A, n=1 << 40):
        if gated:
            return f(dy, xq, xs, wq, sw, b, dx, dw, db, M, N, K, act, w, n, None)
        return f(dy, xq, xs, wq, sw, dx, dw, db, M, N, K, w, n, None)

    for M, N, K in [(-1, 8, 64), (4, 0, 64), (4, 8, 8), (4, 8, 72), (4, 8, 133152), (4, 2 ** 21 + 1, 64),
                    (2 ** 21 + 1, 8, 64)]:
        assert call(M=M, N=N, K=K) == SHAPE, (M, N, K)
    assert call(dy=None) == NULL and call(wq=None) == NULL and call(sw=None) == NULL
    assert call(xq=None) == NULL and call(xs=None) == NULL and call(w=None) == NULL
    assert call(dy=A + 1) == ALIGN and call(dx=A + 1) == ALIGN and call(dw=A + 1) == ALIGN
    assert call(xq=A + 2) == ALIGN and call(wq=A + 2) == ALIGN and call(xs=A + 1) == ALIGN and call(w=A + 8) == ALIGN
    need = wsf(4, 8, 64, 1, 1, 1)
    assert need > 0 and call(n=0) == ARG
    assert call(dx=None, dw=None, db=None) == 0                 # nothing asked for
    assert call(M=0, dx=None, dw=None, db=None, dy=None) == 0
    if gated:
        assert call(act=2) == ARG and call(b=A + 1) == ALIGN
        # everything is needed for any output
        assert call(xq=None, dw=None) == NULL
    assert wsf(0, 8, 64, 1, 1, 1) == 0 and wsf(4, 8, 65, 1, 1, 1) == 0
    # what one output needs is never more than what all need
    for M, N, K in [(1, 1, 16), (100, 33, 64), (4096, 4096, 4096), (777, 4603, 1168)]:
        every = wsf(M, N, K, 1, 1, 1)
        assert all(wsf(M, N, K, *fl) <= every for fl in [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1)])


def test_rope_refusals(w8):
    def call(q=A, k=A, qw=A, cos=A, sin=A, pos=None, qo=A, ko=A, M=4, P=4, Hq=4, Hk=2, D=64, rot=64, eps=1e-6,
             row=512, head=64):
        return w8.lib.w8a8_qk_norm_rope(q, row, head, k, row, head, qw, A, cos, sin, pos, qo, row, head, ko, row,
                                        head, M, P, Hq, Hk, D, rot, eps, 0, None)

    for kw in [dict(M=-1), dict(Hq=0, Hk=0), dict(Hq=-1), dict(D=8), dict(D=72), dict(D=1040), dict(rot=8),
               dict(rot=80), dict(rot=-16), dict(P=0), dict(P=2 ** 31), dict(M=2 ** 26, Hq=64), dict(Hq=65536)]:
        assert call(**kw) == SHAPE, kw
    assert call(eps=-1.0) == ARG and call(eps=float("nan")) == ARG
    assert call(M=0, q=None) == 0
    for n in ("q", "k", "cos", "sin", "qo", "ko"):
        assert call(**{n: None}) == NULL, n
    for n in ("q", "k", "cos", "sin", "qo", "ko", "qw"):
        assert call(**{n: A + 8}) == ALIGN, n
    assert call(row=516) == ALIGN and call(head=68) == ALIGN and call(pos=A + 2) == ALIGN

    def back(q=A, dq=A, gq=A, gqw=A, w=A, n=1 << 40, M=4, D=64):
        v = (512, 64)
        return w8.lib.w8a8_qk_norm_rope_backward(dq, *v, A, *v, q, *v, A, *v, A, A, A, A, None, gq, *v, A, *v, gqw, A,
                                                 M, 4, 4, 2, D, 64, 1e-6, 0, w, n, None)

    assert back(D=72) == SHAPE and back(q=None) == NULL and back(dq=None) == NULL and back(gq=None) == NULL
    assert back(gqw=A + 2) == ALIGN and back(w=None) == NULL and back(w=A + 8) == ALIGN and back(n=16) == ARG


def test_binding_refuses_before_the_library(w8):
    x, wq, ws = torch.zeros(2, 32, dtype=BF), torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8)
    with pytest.raises(ValueError):
        w8.linear_dynamic(x, wq, ws)                             # not on a device
    with pytest.raises(TypeError):
        w8.linear_dynamic(x.float(), wq, ws)
    with pytest.raises(TypeError):
        w8.gated_linear_dynamic(None, wq, ws)
    with pytest.raises(ValueError):
        w8.gated_linear(wq, ws, wq, ws, act="relu")
    with pytest.raises(ValueError):
        w8.gated_linear_backward(x, wq, ws, wq, ws, act="tanh")
    with pytest.raises(ValueError):
        w8.linear_backward(x[0], wq, ws, wq, ws)
    with pytest.raises(ValueError):
        w8.qk_norm_rope(x, x, None, None, ws, ws)


# ---- the gradients' formulas against differences (64 bits) ----

def differences(f, v, steps=1e-6):
    out = torch.zeros_like(v)
    flat, o = v.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + steps
        hi = float(f())
        flat[i] = keep - steps
        lo = float(f())
        flat[i] = keep
        o[i] = (hi - lo) / (2 * steps)
    return out


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_gradient_formula(kind):
    g = torch.Generator().manual_seed(2)
    M, N, K = 3, 4, 16
    x, w = torch.randn(M, K, generator=g, dtype=ref.F64), torch.randn(2 * N, K, generator=g, dtype=ref.F64) * 0.3
    b, dy = torch.randn(2 * N, generator=g, dtype=ref.F64), torch.randn(M, N, generator=g, dtype=ref.F64)
    one_m, one_n = torch.ones(M, dtype=ref.F64), torch.ones(2 * N, dtype=ref.F64)

    def loss():
        return (ref.gated(x, one_m, w, one_n, b, kind) * dy).sum()

    d = ref.gated_d(dy, x, one_m, w, one_n, b, kind)
    for v, (want, _) in zip((x, w, b), ref.product_grads(d, x, one_m, w, one_n)):
        assert torch.allclose(differences(loss, v), want, rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradient_formula(interleaved):
    g = torch.Generator().manual_seed(4)
    M, H, D, rot = 2, 2, 16, 8
    x, dy = (torch.randn(M, H, D, generator=g, dtype=ref.F64) for _ in range(2))
    w = 1 + 0.3 * torch.randn(D, generator=g, dtype=ref.F64)
    a = torch.rand(M, rot // 2, generator=g, dtype=ref.F64) * 6

    def loss():
        return (ref.norm_rope(x, w, a.cos(), a.sin(), 1e-3, interleaved) * dy).sum()

    dx, dw, _ = ref.norm_rope_grad(dy, x, w, a.cos(), a.sin(), 1e-3, interleaved)
    assert torch.allclose(differences(loss, x), dx, rtol=1e-6, atol=1e-8)
    assert torch.allclose(differences(loss, w), dw, rtol=1e-6, atol=1e-8)


def test_module_construction_checks(w8):
    lin = w8.W8A8Linear(torch.zeros(96, 32, dtype=torch.int8), torch.zeros(96), None)
    with pytest.raises(ValueError):
        w8.W8A8QKV(lin, 5, 3)                                    # 96 rows are not 11 heads
    assert w8.W8A8QKV(lin, 2, 2).heads == (2, 2, 16)
    with pytest.raises(ValueError):
        w8.W8A8GatedMLP(torch.zeros(62, 32, dtype=torch.int8), torch.zeros(62), None, lin, "silu")
    down = w8.W8A8Linear(torch.zeros(32, 48, dtype=torch.int8), torch.zeros(32), None)
    with pytest.raises(ValueError):
        w8.W8A8GatedMLP(lin.wq, lin.w_scale, None, down, "tanh")
    m = w8.W8A8GatedMLP(lin.wq, lin.w_scale, None, down)
    with pytest.raises(TypeError):
        m(torch.zeros(2, 32))                                    # bf16 activations only
    assert set(m.state_dict()) == {"wq", "w_scale", "down.wq", "down.w_scale"}


def test_native_calls_leave_everything_unusual_to_the_checks(w8):
    from w8a8_int8_quantized_token_amd import _calls
    x, wq, ws = torch.zeros(2, 32, dtype=BF), torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8)
    q = torch.zeros(2, 2, 16, dtype=BF)
    for args in ((x, wq, ws, None, 0, 1), (None, wq, ws, None, 0, 1), (x, wq, ws, None, 0), (x, wq, ws, None, "a", 1),
                 (x, wq, ws, None, 2 ** 40, 1), (x[0], wq, ws, None, 0, 1), ()):
        assert _calls.dynamic(*args) is None
    assert _calls.backward(x, wq, ws, wq, ws, None, -1, True, True, True) is None
    assert _calls.backward(x, wq, ws, wq, ws, None, -1, 1, True, True) is None
    assert _calls.qk_norm_rope(q, q, None, None, ws, ws, None, "eps", False) is None
    assert _calls.qk_norm_rope_backward(q, q, None, None, x, x, None, 1e-6, False, q, q, True) is None
