"""The linear with low-rank adapters where it can go wrong: values of an
adapter that are not finite, what the other tokens are, and the roundings of
gradients whatever the number of tokens."""
import pytest
import torch

import adapter_ref as aref
import block_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    import w8a8_int8_quantized_token_amd as pkg
    return pkg


def dev(*ts):
    return tuple(None if t is None else t.to(DEV) for t in ts)


def same(a, b):
    a, b = a.detach().contiguous(), b.detach().contiguous()
    return a.shape == b.shape and torch.equal(a.view(torch.int16), b.view(torch.int16))


def inputs(M, K, N, R, L, seed):
    g = torch.Generator().manual_seed(seed + M + N)
    xq, xs = ref.codes_of(torch.randn(M, K, generator=g).to(BF))
    wq, ws = ref.codes_of((torch.randn(N, K, generator=g) * 0.05).to(BF))
    a = (torch.randn(L, R, K, generator=g) / K ** 0.5).to(BF)
    b = (torch.randn(L, N, R, generator=g) * 0.3).to(BF)
    scaling = torch.rand(L, generator=g) + 0.5
    ids = torch.randint(-1, L, (M,), generator=g).to(torch.int32)
    return xq, xs, wq, ws, a, b, ids, scaling


@pytest.mark.parametrize("M,N,K,R", [(1, 300, 256, 16), (5, 300, 1024, 24), (16, 5000, 800, 16), (32, 520, 512, 40), (48, 256, 6144, 16),
                                     (300, 520, 256, 24), (777, 603, 400, 40), (700, 1032, 512, 128), (4608, 4104, 256, 16)])
def test_a_channel_that_is_not_finite_is_alone(w8, M, N, K, R):
    """A NaN or an infinity in an adapter's b reaches its own tokens in its own channel, in every tile alike."""
    xq, xs, wq, ws, a, b, ids, scaling = inputs(M, K, N, R, 4, 1)
    ids[0] = 1
    bad = b.clone()
    bad[1, 5, 2], bad[1, N - 1, R - 1], bad[2, 70, :], bad[3, 200, 0] = INF, NAN, -INF, -INF
    hit = torch.zeros(M, N, dtype=torch.bool)
    for i, n in [(1, 5), (1, N - 1), (2, 70), (3, 200)]:
        hit[ids == i, n] = True
    hit = hit.to(DEV)
    first = dev(xq, xs, wq, ws, a)
    last = dev(ids, scaling)
    for tile in (-1, *range(w8.num_tiles())):
        clean = w8.linear_adapters(*first, b.to(DEV), *last, tile=tile)
        y = w8.linear_adapters(*first, bad.to(DEV), *last, tile=tile)
        assert not torch.isfinite(y[hit]).any(), tile
        assert same(y[~hit], clean[~hit]), tile
        assert torch.isinf(y[(ids == 1).to(DEV), 5]).all() and torch.isinf(y[(ids == 3).to(DEV), 200]).all(), tile


@pytest.mark.parametrize("M,N,K,R", [(5, 64, 300 * 16, 16), (40, 2776, 2592, 16), (300, 520, 272, 24), (700, 2048, 512, 40)])
def test_a_column_that_is_not_finite_is_alone_in_gradients(w8, M, N, K, R):
    """The same of a and the input's gradient."""
    xq, xs, wq, ws, a, b, ids, scaling = inputs(M, K, N, R, 4, 2)
    dy = torch.randn(M, N, generator=torch.Generator().manual_seed(M)).to(BF)
    bad = a.clone()
    bad[1, 2, 5], bad[2, R - 1, K - 1] = INF, NAN
    hit = torch.zeros(M, K, dtype=torch.bool)
    hit[ids == 1, 5] = hit[ids == 2, K - 1] = True
    hit = hit.to(DEV)
    args = dev(dy, xq, xs, wq, ws)
    clean = w8.linear_adapters_backward(*args, *dev(a, b, ids, scaling), da=False, db=False)[0]
    dx = w8.linear_adapters_backward(*args, *dev(bad, b, ids, scaling), da=False, db=False)[0]
    assert not torch.isfinite(dx[hit]).any() and same(dx[~hit], clean[~hit])


@pytest.mark.parametrize("M,K,R", [(4096, 4096, 16), (8192, 4096, 16), (3000, 2576, 32), (2048, 4096, 64)])
def test_a_token_does_not_depend_on_its_neighbours_adapters(w8, M, K, R):
    """t as it is: the weight adds nothing and b is the identity.  Of the gradients, u likewise."""
    L = 16
    xq, xs, _, _, a, _, ids, scaling = inputs(M, K, R, R, L, 3)
    other = torch.where(torch.rand(M, generator=torch.Generator().manual_seed(4)) < 0.5, ids, (ids + 5) % L).to(torch.int32)
    keep = (other == ids).to(DEV)
    runs = torch.arange(M, dtype=torch.int32) * L // M
    no_weight = dev(torch.zeros(R, K, dtype=torch.int8), torch.zeros(R))
    eye = torch.eye(R).to(BF).expand(L, R, R).contiguous()

    def t(ids):
        return w8.linear_adapters(*dev(xq, xs), *no_weight, *dev(a, eye, ids, scaling))

    assert same(t(ids)[keep], t(other)[keep])
    own = (runs == ids).to(DEV)
    assert own.any() and same(t(ids)[own], t(runs)[own])
    dy = torch.randn(M, K, generator=torch.Generator().manual_seed(5)).to(BF)
    b = (a.transpose(1, 2) * 0.3).contiguous()
    no_weight = dev(torch.zeros(K, R, dtype=torch.int8), torch.zeros(K))

    def u(ids):
        return w8.linear_adapters_backward(dy.to(DEV), None, None, *no_weight, *dev(eye, b, ids, scaling), da=False, db=False)[0]

    assert same(u(ids)[keep], u(other)[keep]) and same(u(ids)[own], u(runs)[own])


def rms(e):
    return float(e.square().mean().sqrt())


def once(got, want, rows=None):
    """Beside its own rounding to bf16 no other error of a gradient is seen (fp32 sums, operands to 2^-17)."""
    got, want = got.cpu().double(), want.cpu()
    if rows is not None:
        got, want = got[rows], want[rows]
    return rms(got - want) <= 1.03 * rms(want.to(BF).double() - want)


# few tokens of each adapter in a batch of some, of few assigned tokens among many, of long lists; rows and blocks
# of the first products
ONCE = [(150, 256, 264, 8, 8, "mixed"), (33, 512, 264, 64, 5, "mixed"), (300, 256, 255, 16, 40, "mixed"), (1500, 512, 520, 24, 200, "mixed"),
        (600, 512, 520, 16, 3, "rare"), (2500, 512, 520, 16, 3, "rare"), (2100, 512, 264, 128, 2, "rare"),
        (1000, 512, 520, 16, 1, "mixed"), (4096, 512, 520, 16, 1, "mixed"), (4096, 256, 264, 64, 4, "mixed"), (9000, 256, 136, 32, 2, "mixed"),
        (700, 256, 5, 40, 2, "mixed")]


@pytest.mark.parametrize("M,K,N,R,L,kind", ONCE)
def test_adapters_gradients_are_rounded_once(w8, M, K, N, R, L, kind):
    xq, xs, wq, ws, a, b, ids, scaling = inputs(M, K, N, R, L, 6)
    g = torch.Generator().manual_seed(M)
    dy = torch.randn(M, N, generator=g).to(BF)
    if kind == "rare":
        ids = torch.where(torch.rand(M, generator=g) < 12 / M, ids, torch.full_like(ids, -1))
    inp = (dy, xq, xs, wq, ws, a, b, ids, scaling)
    got = w8.linear_adapters_backward(*dev(*inp))
    want = aref.grads(*inp)
    for i in (1, 2):
        assert once(got[i], want[i][0]), ("da", "db")[i - 1]
    # each asked for alone has the same bits
    assert same(w8.linear_adapters_backward(*dev(*inp), False, True, False)[1], got[1])
    assert same(w8.linear_adapters_backward(*dev(*inp), False, False, True)[2], got[2])


@pytest.mark.parametrize("M", [40, 3000])
def test_infinities_beside_the_roundings_rest(w8, M):
    """An infinity in dy, x's scale or the scaling is no NaN in the gradients that the definition leaves infinite."""
    K, N, R = 64, 136, 16
    xq, xs, wq, ws, a, b, ids, scaling = inputs(M, K, N, R, 2, 7)
    ids = torch.arange(M, dtype=torch.int32) * 2 // M
    dy = torch.randn(M, N, generator=torch.Generator().manual_seed(M)).to(BF)
    plain = w8.linear_adapters_backward(*dev(dy, xq, xs, wq, ws, a, b, ids, scaling))
    bad = dy.clone()
    bad[0, 3], bad[M - 1, 77] = INF, -INF
    got = w8.linear_adapters_backward(*dev(bad, xq, xs, wq, ws, a, b, ids, scaling))[2]
    hit = torch.zeros(2, N, dtype=torch.bool, device=DEV)
    hit[0, 3] = hit[1, 77] = True
    assert torch.isinf(got[hit]).all() and same(got[~hit], plain[2][~hit])
    # an infinite scaling: t is infinite, and db where dy is not zero (a sum of infinities of either sign is a NaN)
    big = scaling.clone()
    big[0] = INF
    one = ids.clone()
    one[1:] = 1                                       # the first adapter has one token
    got = w8.linear_adapters_backward(*dev(dy, xq, xs, wq, ws, a, b, one, big))
    assert torch.isinf(got[2][0]).all() and torch.isfinite(got[2][1].float()).all() and torch.isfinite(got[1][1].float()).all()
    assert torch.isinf(got[1][0][:, (xq[0] != 0).to(DEV)]).all()


@pytest.mark.parametrize("M,R", [(1280, 8), (1281, 8), (1280, 16), (1281, 16), (512, 32), (513, 32), (341, 48), (342, 48), (128, 128), (129, 128)])
def test_gradients_on_both_sides_of_the_first_products_rule(w8, M, R):
    xq, xs, wq, ws, a, b, ids, scaling = inputs(M, 272, 264, R, 3, 8)
    dy = torch.randn(M, 264, generator=torch.Generator().manual_seed(M)).to(BF)
    inp = (dy, xq, xs, wq, ws, a, b, ids, scaling)
    for g, (want, off), name in zip(w8.linear_adapters_backward(*dev(*inp)), aref.grads(*inp), ("dx", "da", "db")):
        ref.check(g, want, off, name, rms_steps=2.0)


def test_more_workgroups_than_a_row_of_the_grid(w8):
    """65536 adapters beside 2184 channels, a few of them with tokens."""
    M, K, N, R, L = 70, 64, 2184, 8, 65536
    g = torch.Generator().manual_seed(9)
    xq, xs = ref.codes_of(torch.randn(M, K, generator=g).to(BF))
    dy = torch.randn(M, N, generator=g).to(BF)
    used = torch.tensor([0, 1, 60000, 65534, 65535])
    ids = used[torch.randint(0, 5, (M,), generator=g)].to(torch.int32)
    a = (torch.randn(5, R, K, generator=g) / K ** 0.5).to(BF)
    scaling = torch.rand(L, generator=g) + 0.5
    all_a = torch.zeros(L, R, K, dtype=BF, device=DEV)
    all_a[used.to(DEV)] = a.to(DEV)
    all_b = torch.zeros(L, N, R, dtype=BF, device=DEV)
    wq, ws = torch.zeros(N, K, dtype=torch.int8), torch.zeros(N)
    db = w8.linear_adapters_backward(*dev(dy, xq, xs, wq, ws), all_a, all_b, *dev(ids, scaling), dx=False, da=False)[2]
    which = torch.stack([(used == int(i)).nonzero()[0, 0] for i in ids]).to(torch.int32)
    want, off = aref.grads(dy, xq, xs, wq, ws, a, torch.zeros(5, N, R, dtype=BF), which, scaling[used])[2]
    ref.check(db[used.to(DEV)], want, off, "db", rms_steps=2.0)
    rest = torch.ones(L, dtype=torch.bool, device=DEV)
    rest[used.to(DEV)] = False
    assert not db[rest].any()
