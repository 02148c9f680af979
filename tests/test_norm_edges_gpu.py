"""The norm that leaves codes, and its gradient, at values where it can go
wrong: NaNs and infinities among the inputs, which no finite result may hide,
and rows whose squares fp32 does not hold."""
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


# squares that vanish or overflow in fp32: rows of these magnitudes
FAR = [2.0 ** e for e in (-132, -126, -110, -90, -74, -70, -64, -52, -48, 0, 50, 62, 66, 90, 120)]


def far_rows(K, seed):
    x = torch.randn(len(FAR), K, generator=torch.Generator().manual_seed(seed)).clamp(-4, 4)
    x[x.abs() < 2.0 ** -6] = 2.0 ** -6
    return (x * torch.tensor(FAR)[:, None]).to(BF)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-33, 1e-30, 1e-12, 1e-6])
@pytest.mark.parametrize("copies,K", [(1, 64), (300, 512), (1, 2064), (1, 4096), (1, 8192), (1, 16400)])
def test_rows_whose_squares_leave_the_range(w8, copies, K, eps, fp8):
    x = far_rows(K, K).repeat(copies, 1)
    w = (1 + 0.3 * torch.randn(K, generator=torch.Generator().manual_seed(1))).clamp(0.25, 2).to(BF)
    q, s, _ = w8.add_rms_norm_quantize(*dev(x, None, w), eps=eps, fp8=fp8)
    eps = float(torch.tensor(eps))              # as the kernel has it
    want_q, want_s, _ = aref.norm_codes(x, None, w, eps, fp8)
    assert torch.equal((fp8_values(q) if fp8 else q.float()).cpu(), want_q)
    # the bound of the ordinary rows' test, and half a step of the smallest fp32 number
    assert ((s.cpu().double() - want_s).abs() <= ((64 + 6 + 16 + 2) / 2 + 4) * U * want_s + 2.0 ** -150).all()


@pytest.mark.parametrize("eps", [0.0, 1e-33, 1e-6])
@pytest.mark.parametrize("copies,K", [(1, 64), (280, 512), (1, 2064), (1, 4096), (1, 8192), (1, 16384), (1, 16400)])
def test_gradient_of_rows_whose_squares_leave_the_range(w8, copies, K, eps):
    h = far_rows(K, K + 1).repeat(copies, 1)
    M = h.shape[0]
    g = torch.Generator().manual_seed(2)
    w = (1 + 0.3 * torch.randn(K, generator=g)).clamp(0.25, 2).to(BF)
    dn = (torch.randn(M, K, generator=g) * 2.0 ** -20).to(BF)
    dh = torch.randn(M, K, generator=g).to(BF)
    for other in (None, dh):
        dx, dw = w8.add_rms_norm_backward(*dev(dn, h, w), eps=eps, dh=None if other is None else other.to(DEV))
        want, size, want_dw, dw_size = aref.norm_grad(dn, other, h, w, float(torch.tensor(eps)))
        # (the ordinary rows' bounds; row by row, since magnitudes differ)
        off = (dx.cpu().double() - want).abs()
        assert (off <= 2 * (64 + 22 + 8) * U * size + 2.0 ** -8 * want.abs() + 2.0 ** -134).all()
        assert ((dw.cpu().double() - want_dw).abs() <= (M + 64 + 60) * U * dw_size + 1e-30).all()


@pytest.mark.parametrize("K", [512, 2064, 4096, 8192, 12288, 20480])
def test_gradient_of_such_rows_in_place(w8, K):
    h = far_rows(K, 5).repeat(90, 1)
    dn, dh = (torch.randn_like(h.float()).mul(2.0 ** -20).to(BF) for _ in range(2))
    want = w8.add_rms_norm_backward(*dev(dn, h), eps=0.0, dh=dh.to(DEV))
    for into in range(3):
        t = list(dev(dn, h, dh))
        got = w8.add_rms_norm_backward(t[0], t[1], eps=0.0, dh=t[2], dx=t[into])
        assert got[0].data_ptr() == t[into].data_ptr()
        assert torch.equal(bits(got[0]), bits(want[0])) and torch.equal(bits(got[1]), bits(want[1]))


def test_zero_rows_pass_the_residuals_gradient_alone(w8):
    z = torch.zeros(3, 2064, dtype=BF, device=DEV)
    dx, dw = w8.add_rms_norm_backward(z + 1, z, None, eps=0.0, dh=z + 2)
    assert (dx == 2).all() and not dw.any()
    q, s, _ = w8.add_rms_norm_quantize(z, eps=0.0)
    assert not q.any() and not s.any()


# both sides of the sizes at which the gradient's workgroups change
@pytest.mark.parametrize("M,K", [(1024, 2048), (1024, 2064), (1025, 2064), (1500, 3568), (1500, 3584), (100, 3568), (1030, 4080), (1030, 4112)])
def test_gradient_on_both_sides_of_its_rules(w8, M, K):
    h, dh, w = inputs(M, K, 3)
    dn = torch.randn(M, K, generator=torch.Generator().manual_seed(K)).to(BF)
    dx, dw = w8.add_rms_norm_backward(*dev(dn, h, w), eps=1e-5, dh=dh.to(DEV))
    want, size, want_dw, dw_size = aref.norm_grad(dn, dh, h, w, 1e-5)
    ref.check(dx, want, 2 * (64 + 22 + 8) * U * size, "dx")
    assert ((dw.cpu().double() - want_dw).abs() <= (M + 64 + 60) * U * dw_size + 1e-30).all()
    need = w8.lib.w8a8_add_rms_norm_backward_workspace(M, K)
    space = torch.full((need + 32,), 255, dtype=torch.uint8, device=DEV)
    got = w8.add_rms_norm_backward(*dev(dn, h, w), eps=1e-5, dh=dh.to(DEV), workspace=space[:need])
    assert torch.equal(bits(got[0]), bits(dx)) and torch.equal(bits(got[1]), bits(dw)) and (space[need:] == 255).all()
