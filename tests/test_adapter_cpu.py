"""Host-side checks of the norm that leaves codes and of the adapters: refusals
before any launch (fake pointers, never dereferenced), the binding's argument
checks, and the formulas that the GPU tests compare with, against differences."""
import pytest
import torch

import adapter_ref as aref
import block_ref as ref

A = 0x10000
BF = torch.bfloat16
NULL, SHAPE, ALIGN, ARG = 1, 2, 3, 5


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_quantized_token_amd as pkg
    return pkg


def test_norm_refusals(w8):
    def call(x=A, r=A, w=A, h=A, q=A, s=A, M=4, K=64, eps=1e-6, fp8=0):
        return w8.lib.w8a8_add_rms_norm_quantize(x, r, w, h, q, s, M, K, eps, fp8, None)

    def back(dn=A, dh=A, h=A, w=A, dx=A, dw=A, M=4, K=64, eps=1e-6, ws=A, n=1 << 40):
        return w8.lib.w8a8_add_rms_norm_backward(dn, dh, h, w, dx, dw, M, K, eps, ws, n, None)

    size = w8.lib.w8a8_add_rms_norm_backward_workspace
    for M, K in [(-1, 64), (4, 0), (4, 8), (4, 24), (4, 32784), (2 ** 26 + 1, 16), (2 ** 26, 16), (2 ** 24, 8192), (2 ** 22, 32768)]:
        assert call(M=M, K=K) == SHAPE and back(M=M, K=K) == SHAPE and size(M, K) == 0, (M, K)
    for eps in (-1.0, float("nan")):
        assert call(eps=eps) == ARG and back(eps=eps) == ARG
    assert call(M=0, x=None) == 0 and back(M=0, dn=None, dw=None) == 0
    for n in ("x", "q", "s"):
        assert call(**{n: None}) == NULL, n
    for n in ("dn", "h", "dx", "ws"):
        assert back(**{n: None}) == NULL, n
    for n in ("x", "r", "w", "h", "q"):
        assert call(**{n: A + 8}) == ALIGN, n
    for n in ("dn", "dh", "h", "w", "dx", "ws"):
        assert back(**{n: A + 8}) == ALIGN, n
    assert call(s=A + 2) == ALIGN and back(dw=A + 2) == ALIGN and back(n=16) == ARG
    assert size(4, 64) >= 4 * 64 and size(100000, 4096) < 100000 * 4096


def test_adapter_refusals(w8):
    def codes(xq=A, xs=A, wq=A, sw=A, bias=A, a=A, b=A, sc=A, ids=A, y=A, M=4, N=8, K=64, R=16, L=3, tile=-1, ws=A, n=1 << 40):
        return w8.lib.w8a8_linear_adapters(xq, xs, wq, sw, bias, a, b, sc, ids, y, M, N, K, R, L, tile, ws, n, None)

    def dynamic(x=A, wq=A, sw=A, bias=A, a=A, b=A, sc=A, ids=A, y=A, M=40, N=8, K=64, R=16, L=3, ws=A, n=1 << 40):
        return w8.lib.w8a8_linear_adapters_dynamic(x, wq, sw, bias, a, b, sc, ids, y, M, N, K, R, L, ws, n, None)

    size = w8.lib.w8a8_linear_adapters_workspace
    for bad in [dict(M=-1), dict(N=0), dict(K=0), dict(K=24), dict(K=133152), dict(M=2 ** 26 + 1), dict(N=2 ** 26 + 1), dict(R=0),
                dict(R=4), dict(R=12), dict(R=136), dict(L=0), dict(L=65537), dict(R=-8)]:
        assert codes(**bad) == SHAPE and dynamic(**bad) == SHAPE, bad
    assert codes(M=0, xq=None, y=None) == 0 and dynamic(M=0, x=None, ws=None, n=0) == 0
    for n in ("xq", "xs", "wq", "sw", "a", "b", "sc", "ids", "y", "ws"):
        assert codes(**{n: None}) == NULL, n
    for n in ("x", "wq", "sw", "a", "b", "sc", "ids", "y", "ws"):
        assert dynamic(**{n: None}) == NULL, n
    for n in ("xq", "wq", "a", "b", "ws"):
        assert codes(**{n: A + 8}) == ALIGN, n
    for n in ("xs", "sw", "sc", "ids"):
        assert codes(**{n: A + 2}) == ALIGN, n
    assert codes(y=A + 1) == ALIGN and codes(bias=A + 1) == ALIGN and dynamic(x=A + 2) == ALIGN
    assert codes(tile=w8.num_tiles()) == ARG
    assert codes(n=4 * 16 * 2 - 1) == ARG and dynamic(n=16) == ARG
    assert size(4, 8, 64, 16, 0) >= 4 * 16 * 2 and size(40, 8, 64, 16, 1) >= 40 * (16 * 2 + 64 + 4)
    assert size(4, 8, 64, 12, 0) == 0 and size(0, 8, 64, 16, 1) == 0
    # one token makes its codes and first products in the kernel itself
    assert size(1, 2048, 2048, 16, 1) == 0 and size(1, 2048, 2048, 128, 1) > 0


def test_adapter_backward_refusals(w8):
    def call(dy=A, xq=A, xs=A, wq=A, sw=A, a=A, b=A, sc=A, ids=A, dx=A, da=A, db=A, M=4, N=8, K=64, R=16, L=3, ws=A, n=1 << 40):
        return w8.lib.w8a8_linear_adapters_backward(dy, xq, xs, wq, sw, a, b, sc, ids, dx, da, db, M, N, K, R, L, ws, n, None)

    size = w8.lib.w8a8_linear_adapters_backward_workspace
    for bad in [dict(M=-1), dict(N=0), dict(K=24), dict(K=133152), dict(R=4), dict(R=136), dict(L=0), dict(L=65537),
                dict(N=2 ** 21 + 1), dict(K=133136, N=2 ** 20, L=65536, R=128)]:
        assert call(**bad) == SHAPE, bad
    assert call(dx=None, da=None, db=None) == 0 and call(M=0, dx=None, da=None, db=None, dy=None) == 0
    for n in ("dy", "xq", "xs", "wq", "sw", "a", "b", "sc", "ids", "ws"):
        assert call(**{n: None}) == NULL, n
    # what an output does not need may be missing
    assert call(xq=None, da=None) == NULL and call(wq=None, dx=None, ws=None) == NULL
    for n in ("xq", "wq", "a", "b", "da", "db", "ws"):
        assert call(**{n: A + 8}) == ALIGN, n
    for n in ("xs", "sw", "sc", "ids"):
        assert call(**{n: A + 2}) == ALIGN, n
    assert call(dy=A + 1) == ALIGN and call(dx=A + 1) == ALIGN and call(n=16) == ARG
    every = size(100, 72, 64, 16, 3, 1, 1, 1)
    for fl in [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1)]:
        assert 0 < size(100, 72, 64, 16, 3, *fl) <= every
    assert size(0, 72, 64, 16, 3, 1, 1, 1) == 0 and size(4, 72, 64, 12, 3, 1, 1, 1) == 0


def test_binding_refuses_before_the_library(w8):
    x, wq, ws = torch.zeros(2, 32, dtype=BF), torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8)
    a, b = torch.zeros(3, 8, 32, dtype=BF), torch.zeros(3, 8, 8, dtype=BF)
    ids, sc = torch.zeros(2, dtype=torch.int32), torch.zeros(3)
    xq, xs = torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2)
    with pytest.raises(ValueError):
        w8.linear_adapters_dynamic(x, wq, ws, a, b, ids, sc)         # not on a device
    with pytest.raises(ValueError):
        w8.linear_adapters(xq, xs, wq, ws, a, b, ids, sc)
    with pytest.raises(ValueError):
        w8.linear_adapters_backward(torch.zeros(2, 8, dtype=BF), xq, xs, wq, ws, a, b, ids, sc)
    with pytest.raises(ValueError):
        w8.add_rms_norm_quantize(x)
    with pytest.raises(ValueError):
        w8.add_rms_norm_backward(x, x)
    for f in (lambda: w8.linear_adapters_dynamic(x.float(), wq, ws, a, b, ids, sc),
              lambda: w8.linear_adapters_dynamic(None, wq, ws, a, b, ids, sc),
              lambda: w8.linear_adapters(x, xs, wq, ws, a, b, ids, sc),
              lambda: w8.add_rms_norm_quantize(x.half()), lambda: w8.add_rms_norm_backward(x, None)):
        with pytest.raises(TypeError):
            f()


# ---- the formulas ----

def test_norm_codes_stand_for_the_normed_row():
    """code * scale is the normed value to within half a code's step (and the fp32 roundings of s and v / s)."""
    g = torch.Generator().manual_seed(0)
    x, r, w = (torch.randn(*s, generator=g).to(BF) for s in ((20, 96), (20, 96), (96,)))
    for fp8 in (False, True):
        q, s, h = aref.norm_codes(x, r, w, 1e-6, fp8)
        n = h.double() / (h.double().square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
        step = s[:, None] if not fp8 else (q.abs().double() * 2 ** -3 + 2 ** -9) * s[:, None]
        assert ((q.double() * s[:, None] - n).abs() <= step * (0.5 + 2 ** -15)).all()
        assert q.abs().amax(1).eq(448 if fp8 else 127).all()


def test_norm_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(1)
    h, dn, dh, w = (torch.randn(*s, generator=g).to(BF) for s in ((4, 16), (4, 16), (4, 16), (16,)))
    dx, _, dw, _ = aref.norm_grad(dn, dh, h, w, 1e-3)
    h64, w64 = h.double().requires_grad_(), w.double().requires_grad_()
    n = h64 / (h64.square().mean(1, keepdim=True) + 1e-3).sqrt() * w64
    ((n * dn.double()).sum() + (h64 * dh.double()).sum()).backward()
    assert torch.allclose(dx, h64.grad, atol=1e-12) and torch.allclose(dw, w64.grad, atol=1e-12)


def test_adapter_formulas_against_differences():
    g = torch.Generator().manual_seed(2)
    M, K, N, R, L = 9, 16, 12, 8, 3
    xq, xs = ref.codes_of(torch.randn(M, K, generator=g).to(BF))
    wq, ws = ref.codes_of(torch.randn(N, K, generator=g).to(BF))
    a, b = torch.randn(L, R, K, generator=g).to(BF), torch.randn(L, N, R, generator=g).to(BF)
    sc, ids = torch.randn(L, generator=g), torch.randint(-1, L + 1, (M,), generator=g)
    dy = torch.randn(M, N, generator=g).to(BF)
    x = (xq.double() * xs.double()[:, None]).requires_grad_()
    a64, b64 = a.double().requires_grad_(), b.double().requires_grad_()
    y = x @ (wq.double() * ws.double()[:, None]).T
    rows = []
    for m in range(M):
        i = int(ids[m])
        add = sc[i].double() * b64[i] @ (a64[i] @ x[m]) if 0 <= i < L else 0
        rows.append(y[m] + add)
    y = torch.stack(rows)
    got, _ = aref.linear(xq, xs, wq, ws, a, b, ids, sc, None)
    assert torch.allclose(got, y.detach(), atol=1e-10)
    (y * dy.double()).sum().backward()
    for (want, off), t in zip(aref.grads(dy, xq, xs, wq, ws, a, b, ids, sc), (x, a64, b64)):
        assert torch.allclose(want, t.grad, atol=1e-9) and (off >= 0).all()
