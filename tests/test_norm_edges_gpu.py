"""The norm that leaves codes, and its gradient, at values where it can go
wrong: NaNs and infinities among the inputs, which no finite result may hide."""
import pytest
import torch

import adapter_ref as aref
import block_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16
U = aref.U
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    import w8a8_int8_quantized_token_amd as pkg
    return pkg


def dev(*ts):
    return tuple(None if t is None else t.to(DEV) for t in ts)


def bits(t):
    return t.detach().contiguous().view(torch.uint8).cpu()


def inputs(M, K, seed=0):
    g = torch.Generator().manual_seed(seed + M + K)
    return (torch.randn(M, K, generator=g).to(BF), torch.randn(M, K, generator=g).to(BF),
            (1 + 0.3 * torch.randn(K, generator=g)).to(BF))


def fp8_values(q):
    return q.view(torch.float8_e4m3fn).float()


# one, four and sixteen wavefronts to a row, several rows to a workgroup
SIZES = [(8, 512), (4100, 512), (9, 2064), (4099, 528), (8, 8192)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_what_is_not_finite_reaches_the_scale(w8, M, K, fp8):
    """A row with a NaN or an infinity has a scale that is not finite, as quantize_act's; others keep their bits."""
    x, r, w = inputs(M, K)
    clean = w8.add_rms_norm_quantize(*dev(x, r, w), fp8=fp8)
    bx, br = x.clone(), r.clone()
    bx[0] = NAN
    bx[1, K - 1] = NAN
    br[2, 5] = NAN
    bx[3, 7] = INF
    bx[4, 8], br[4, 8] = INF, -INF
    bx[5, 1], br[M - 1, K // 2] = -INF, NAN
    rows = torch.tensor([0, 1, 2, 3, 4, 5, M - 1])
    others = torch.ones(M, dtype=torch.bool)
    others[rows] = False
    for weight in (w, None):
        q, s, h = w8.add_rms_norm_quantize(*dev(bx, br, weight), fp8=fp8)
        assert torch.isnan(s[rows.to(DEV)]).all()
        assert torch.isfinite(s[others.to(DEV)]).all()
        if weight is not None:
            for got, want in zip((q, s, h), clean):
                assert torch.equal(bits(got[others.to(DEV)]), bits(want[others.to(DEV)]))
    # no linear after it sees a finite row
    if not fp8:
        wq, ws = w8.quantize_weight(torch.randn(24, K, device=DEV).to(BF))
        assert not torch.isfinite(w8.linear(q, s, wq, ws).float()[rows.to(DEV)]).any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_weights_that_are_not_finite(w8, M, K, fp8):
    x, _, w = inputs(M, K)
    for at, value in [(slice(None), NAN), (K - 3, NAN), (1, INF), (K // 2, -INF)]:
        bad = w.clone()
        bad[at] = value
        _, s, _ = w8.add_rms_norm_quantize(*dev(x, None, bad), fp8=fp8)
        assert not torch.isfinite(s).any(), (at, value)
    # an infinity times a zero of the weight is a NaN; finite rows times zeros are zeros
    zero = w.clone()
    zero[3] = 0
    bx = x.clone()
    bx[2, 3] = INF
    _, s, _ = w8.add_rms_norm_quantize(*dev(bx, None, zero), fp8=fp8)
    assert torch.isnan(s[2]) and torch.isfinite(s[torch.arange(M, device=DEV) != 2]).all()
    q, s, _ = w8.add_rms_norm_quantize(*dev(x, None, torch.zeros_like(w)), fp8=fp8)
    assert not s.any() and not (fp8_values(q) if fp8 else q).any()


# every form of the gradient's rows, with and without the next row's loads ahead
GRADS = [(5, 512), (6, 2064), (5, 4096), (4, 8192), (4, 12288), (3, 20480)]


@pytest.mark.parametrize("M,K", GRADS)
def test_gradient_of_rows_that_are_not_finite(w8, M, K):
    h, dh, w = inputs(M, K, 1)
    dn = torch.randn(M, K, generator=torch.Generator().manual_seed(K)).to(BF)
    clean = w8.add_rms_norm_backward(*dev(dn, h, w), dh=dh.to(DEV))
    bad = h.clone()
    bad[1, K - 2] = NAN
    dx, dw = w8.add_rms_norm_backward(*dev(dn, bad, w), dh=dh.to(DEV))
    keep = torch.arange(M, device=DEV) != 1
    assert torch.isnan(dx[1]).all() and torch.equal(bits(dx[keep]), bits(clean[0][keep]))
    assert torch.isnan(dw).all()                # hh is a NaN in the whole row
    bad = dn.clone()
    bad[2, 3] = NAN
    dx, dw = w8.add_rms_norm_backward(*dev(bad, h, w), dh=dh.to(DEV))
    keep = torch.arange(M, device=DEV) != 2
    assert torch.isnan(dx[2]).all() and torch.equal(bits(dx[keep]), bits(clean[0][keep]))
    cols = torch.arange(K, device=DEV) != 3
    assert torch.isnan(dw[3]) and torch.equal(bits(dw[cols]), bits(clean[1][cols]))
    bad = w.clone()
    bad[5] = NAN
    assert torch.isnan(w8.add_rms_norm_backward(*dev(dn, h, bad))[0]).all()
