"""Calls of the operators around the linear at the edges of what their
documentation allows."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    import w8a8_int8_quantized_token_amd as pkg
    return pkg


def same(a, b):
    return torch.equal(a.detach().contiguous().view(torch.int16), b.detach().contiguous().view(torch.int16))


def bf(g, *shape):
    return torch.randn(*shape, generator=g).to(BF).to(DEV)


# ---- padding rows ----

@pytest.mark.parametrize("interleaved", [False, True])
def test_padding_rows_without_a_rotation(w8, interleaved):
    """rot = 0 is the norm alone; rows at a position outside the table are
    padding all the same."""
    M, P, Hq, Hk, D = 37, 50, 6, 2, 128
    g = torch.Generator().manual_seed(1)
    q, k, dq, dk = bf(g, M, Hq, D), bf(g, M, Hk, D), bf(g, M, Hq, D), bf(g, M, Hk, D)
    qw, kw = bf(g, D), bf(g, D)
    none = torch.empty(P, 0, device=DEV)
    pos = torch.randint(0, P, (M,), generator=g, dtype=torch.int32)
    pad = [3, 20, 36]
    pos[3], pos[20], pos[36] = -1, P, 2 ** 31 - 1
    pos = pos.to(DEV)
    keep = [r for r in range(M) if r not in pad]
    room = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    for given in (False, True):      # a plain call and one through the binding's checks
        out = w8.qk_norm_rope(q, k, qw, kw, none, none, pos, interleaved=interleaved,
                              **({"q_out": torch.empty_like(q)} if given else {}))
        want = w8.qk_norm_rope(q, k, qw, kw, none, none, interleaved=interleaved)
        got = w8.qk_norm_rope_backward(dq, dk, q, k, qw, kw, none, none, pos, interleaved=interleaved,
                                       **({"workspace": room} if given else {}))
        part = w8.qk_norm_rope_backward(dq[keep], dk[keep], q[keep], k[keep], qw, kw, none, none,
                                        interleaved=interleaved)
        for i in range(2):
            assert not out[i][pad].any() and same(out[i][keep], want[i][keep])
            assert not got[i][pad].any() and same(got[i][keep], part[i])
            # the same terms in another order: fp32 sums of M heads' products
            assert torch.allclose(got[2 + i], part[2 + i], rtol=1e-4, atol=1e-4 * float(part[2 + i].abs().max()))


@pytest.mark.parametrize("interleaved", [False, True])
def test_padding_rows_are_zeros_whatever_the_tables_hold(w8, interleaved):
    M, P, H, D = 9, 6, 2, 64
    g = torch.Generator().manual_seed(2)
    q, k = bf(g, M, H, D), bf(g, M, H, D)
    cos, sin = torch.rand(P, 16, generator=g).to(DEV), torch.rand(P, 16, generator=g).to(DEV)
    cos[0], sin[0] = float("inf"), float("nan")       # a row that no token is at
    pos = torch.randint(1, P, (M,), generator=g, dtype=torch.int32)
    pos[4], pos[8] = -1, P
    q[4], k[8] = float("nan"), float("inf")
    out = w8.qk_norm_rope(q, k, None, None, cos, sin, pos.to(DEV), interleaved=interleaved)
    back = w8.qk_norm_rope_backward(q, k, q, k, None, None, cos, sin, pos.to(DEV), interleaved=interleaved)
    keep = [0, 1, 2, 3, 5, 6, 7]
    for t in (*out, *back[:2]):
        assert not t[[4, 8]].any() and bool(torch.isfinite(t[keep]).all())
    assert bool(torch.isfinite(back[2]).all()) and bool(torch.isfinite(back[3]).all())
