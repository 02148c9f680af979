"""Gradients and the gated product on inputs whose every operand, product and
sum is exact, so that the results have to be bf16(the 64-bit result) bit for
bit: one summed channel, chunk or row block left out or taken twice changes
them, which a bound of half a bf16 step per term does not see.

Scales are powers of two, codes and dy small integers.  Then dy, codes, their
scaled values and (gated, below) dg and du have at most 8 significant bits and
are exact in bf16, and every partial sum is a whole number, below 2^24, of the
smallest term's unit, so that fp32 sums are exact in any order."""
import pytest
import torch

from test_block_gpu import BACK, TILES

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16
F64 = torch.float64


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    import w8a8_int8_quantized_token_amd as pkg
    return pkg


class Inputs:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV).manual_seed(seed)

    def whole(self, lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=self.g, device=DEV)

    def powers(self, lo, hi, n):
        return 2.0 ** self.whole(lo, hi, n).float()

    def signs(self, share, *shape):
        """-1, 0 or 1, `share` of them not 0."""
        at = torch.rand(shape, generator=self.g, device=DEV) < share
        return (at * (2 * self.whole(0, 1, *shape) - 1)).to(torch.int8)


def whole_sums(terms, unit):
    """The largest sum of magnitudes in units of the smallest term."""
    assert float(terms.max() / unit) < 2 ** 24


def same(got, want, what):
    """got is bf16(want), want exact in fp32."""
    assert torch.equal(want, want.float().to(F64)), what
    want = want.to(BF)
    wrong = (got != want).nonzero()
    assert wrong.numel() == 0, (what, len(wrong), wrong[:4].tolist())


@pytest.mark.parametrize("M,N,K", BACK + TILES)
def test_linear_gradients_exactly(w8, M, N, K):
    r = Inputs(M + 7 * N + K)
    wq, xq = r.whole(-7, 7, N, K).to(torch.int8), r.whole(-7, 7, M, K).to(torch.int8)
    ws, xs = r.powers(-8, -6, N), r.powers(-2, 0, M)
    dy = r.whole(-2, 2, M, N).to(BF)
    d, w, x = dy.to(F64), wq.to(F64) * ws.to(F64)[:, None], xq.to(F64) * xs.to(F64)[:, None]
    whole_sums(d.abs() @ w.abs(), 2.0 ** -8)
    whole_sums(d.abs().T @ x.abs(), 2.0 ** -2)
    dx, dw, db = w8.linear_backward(dy, xq, xs, wq, ws)
    same(dx, d @ w, "dx")
    same(dw, d.T @ x, "dw")
    same(db, d.sum(0), "dbias")
    same(w8.linear_backward(dy, None, None, wq, ws, dw=False, dbias=False)[0], d @ w, "dx alone")


def gated_inputs(M, N, K, act):
    """Inputs with gates from 18 on, where both activations are the identity
    in fp32: 1 + 2^(-18 log2 e) and 1 - erfc(18 / sqrt 2) / 2 round to 1.

    Codes are so few that a sum of K products, 9 of them other than 0 in the
    mean, stays within 23 (checked).  Gates are 64 + halves up to 23 * 2, below
    128: 8 bits.  Up values are quarters within 23 + 4: 8 bits."""
    r = Inputs(M + 3 * N + K + (act == "gelu"))
    share = min(1.0, 3.0 / K ** 0.5)
    wq, xq = r.signs(share, 2 * N, K), r.signs(share, M, K)
    xs = r.powers(-1, 0, M)
    ws = torch.cat([r.powers(0, 1, N), r.powers(-1, 0, N)])
    bias = torch.cat([torch.full((N,), 64.0, device=DEV), r.whole(-4, 4, N).float()])
    dy = r.whole(-2, 2, M, N).to(BF)
    acc = xq.to(F64) @ wq.to(F64).T
    assert float(acc.abs().max()) <= 23
    z = acc * xs.to(F64)[:, None] * ws.to(F64) + bias.to(F64)
    assert float(z[:, :N].min()) >= 18 and float(z[:, :N].max()) < 128
    return dy, xq, xs, wq, ws, bias.to(BF), z


@pytest.mark.parametrize("M,N,K,act", [(*s, ("silu", "gelu")[i % 2]) for i, s in enumerate(BACK + TILES)])
def test_gated_product_and_gradients_exactly(w8, M, N, K, act):
    dy, xq, xs, wq, ws, bias, z = gated_inputs(M, N, K, act)
    same(w8.gated_linear(xq, xs, wq, ws, bias, act=act), z[:, :N] * z[:, N:], "y")
    d = torch.cat([dy.to(F64) * z[:, N:], dy.to(F64) * z[:, :N]], 1)
    w, x = wq.to(F64) * ws.to(F64)[:, None], xq.to(F64) * xs.to(F64)[:, None]
    # dg: quarters, du: halves; times a weight's scale of 1 to 2 and 1/2 to 1,
    # or a token's of 1/2 to 1
    whole_sums(d.abs() @ w.abs(), 0.25)
    whole_sums(d.abs().T @ x.abs(), 0.125)
    whole_sums(d.abs().sum(0), 0.25)
    dx, dw, db = w8.gated_linear_backward(dy, xq, xs, wq, ws, bias, act=act)
    same(dx, d @ w, "dx")
    same(dw, d.T @ x, "dw")
    same(db, d.sum(0), "dbias")
    same(w8.gated_linear_backward(dy, xq, xs, wq, ws, bias, act=act, dw=False, dbias=False)[0], d @ w, "dx alone")
