"""The norm that leaves codes and the linear with low-rank adapters on the GPU
against plain 64-bit forms: sizes from one row on, odd and ragged ones, ids in
any order, rows without an adapter, and adapters that hold NaNs."""
import pytest
import torch

import adapter_ref as aref
import block_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16
U = aref.U


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    import w8a8_int8_quantized_token_amd as pkg
    return pkg


def dev(*ts):
    return tuple(None if t is None else t.to(DEV) for t in ts)


def same(a, b):
    a, b = a.detach().contiguous().cpu(), b.detach().contiguous().cpu()
    if a.dtype == BF:
        a, b = a.view(torch.int16), b.view(torch.int16)
    return a.dtype == b.dtype and torch.equal(a, b)


# ---- norm ----

def norm_inputs(M, K, seed, residual=True, weight=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[:, :: max(K // 8, 1)] *= 20.0
    r = torch.randn(M, K, generator=g).mul(3).to(BF) if residual else None
    w = (1 + 0.3 * torch.randn(K, generator=g)).to(BF) if weight else None
    return x.to(BF), r, w


def fp8_values(q):
    return q.view(torch.float8_e4m3fn).float()


# one row and few, both layouts of many rows, every number of pieces to a lane, the longest
NORMS = [(1, 16), (1, 4096), (3, 528), (5, 4112), (2, 8192), (2, 12288), (2, 12304), (3, 16384), (2, 16400), (2, 32768), (1023, 512),
         (1024, 512), (1025, 528), (1200, 1040), (1027, 2064), (1024, 3088), (1030, 4096), (1100, 16),
         (4097, 16), (4096, 512), (4099, 528), (4098, 1024), (4096, 1040), (512, 4096), (513, 4112), (520, 6160), (40, 8176)]


@pytest.mark.parametrize("M,K", NORMS)
@pytest.mark.parametrize("fp8", [False, True])
def test_norm_codes(w8, M, K, fp8):
    x, r, w = norm_inputs(M, K, M + K)
    for res, wt in [(r, w), (None, w), (r, None), (None, None)]:
        q, s, h = w8.add_rms_norm_quantize(*dev(x, res, wt), eps=1e-5, fp8=fp8)
        want_q, want_s, want_h = aref.norm_codes(x, res, wt, 1e-5, fp8)
        assert q.dtype == (torch.uint8 if fp8 else torch.int8) and s.dtype == torch.float32
        assert same(h, want_h)
        got = (fp8_values(q) if fp8 else q.float()).cpu()
        assert torch.equal(got, want_q)
        # a lane adds at most 64 squares, then 6 exchanges and at most 16 wavefronts; half of that through the
        # root; s, the mean, the root and the quotient round once each
        assert ((s.cpu().double() - want_s).abs() <= ((64 + 6 + 16 + 2) / 2 + 4) * U * want_s).all()


def test_norm_rows_of_zeros_and_small_numbers(w8):
    K = 256
    x = torch.randn(8, K).to(BF)
    x[0] = 0
    x[1] = 0
    x[1, 7] = -2.0 ** -130
    x[2] = torch.randn(K).mul(2.0 ** -70).to(BF)    # squares below the smallest fp32 number
    x[3] = torch.randn(K).mul(2.0 ** 50).to(BF)
    w = torch.ones(K).to(BF)
    w[7] = 2.0 ** -15                               # row 1: a product whose scale is zero
    for eps in (0.0, 1e-6):
        for fp8 in (False, True):
            q, s, _ = w8.add_rms_norm_quantize(*dev(x, None, w), eps=eps, fp8=fp8)
            want_q, want_s, _ = aref.norm_codes(x, None, w, eps, fp8)
            got = (fp8_values(q) if fp8 else q.float()).cpu()
            rows = [0, 1, 3, 4, 5, 6, 7] if eps == 0 else range(8)   # (row 2's squares vanish in fp32)
            for i in rows:
                assert torch.equal(got[i], want_q[i]), i
                if eps > 0 or i != 1:
                    assert abs(float(s[i]) - float(want_s[i])) <= 60 * U * float(want_s[i]), i
            assert not q[0].any() and float(s[0]) == 0 and float(s[1]) == 0
            assert torch.isfinite(s[[0, 1]]).all()


def test_norm_rows_of_subnormal_scales(w8):
    # a scale of one subnormal step stands for a quotient of 1.49 (1.34): codes are clamped, not wrapped
    K = 768
    x, w = torch.zeros(6, K).to(BF), torch.full((K,), 2.0 ** -49).to(BF)
    x[0, 5], x[0, 6], x[0, 700] = 190 * 2.0 ** -100, -190 * 2.0 ** -100, 31 * 2.0 ** -100
    x[1, 5], x[1, 6], x[1, 700] = 600 * 2.0 ** -100, -600 * 2.0 ** -100, 224 * 2.0 ** -100
    x[2, 9] = 300 * 2.0 ** -100
    x[3, 767] = -63 * 2.0 ** -100
    for fp8 in (False, True):
        q, s, _ = w8.add_rms_norm_quantize(*dev(x, None, w), eps=1e-6, fp8=fp8)
        want_q, _, _ = aref.norm_codes(x, None, w, 1e-6, fp8)
        assert torch.equal((fp8_values(q) if fp8 else q.float()).cpu(), want_q)
        assert want_q.abs().max() == (448 if fp8 else 127)
        assert torch.isfinite(s).all()


def test_norm_into_its_inputs_and_as_the_linears_input(w8):
    M, K = 40, 768
    x, r, w = norm_inputs(M, K, 5)
    want = w8.add_rms_norm_quantize(*dev(x, r, w))
    for into in (0, 1):
        t = list(dev(x, r, w))
        q, s, h = w8.add_rms_norm_quantize(*t, h=t[into])
        assert h.data_ptr() == t[into].data_ptr() and all(same(a, b) for a, b in zip((q, s, h), want))
    t = x.to(DEV)
    assert w8.add_rms_norm_quantize(t)[2] is t      # nothing added: h is x
    out = torch.empty_like(t)
    assert same(w8.add_rms_norm_quantize(t, h=out)[2], x) and same(out, x)
    # the normed rows through quantize_act: codes of the bf16-rounded row may differ by one, values by a step
    q, s, h = want
    n = (h.float() * torch.rsqrt(h.float().square().mean(1, keepdim=True) + 1e-6) * w.to(DEV).float()).to(BF)
    q2, s2 = w8.quantize_act(n)
    assert (q.int() - q2.int()).abs().max() <= 1 and ((s - s2).abs() <= 2.0 ** -8 * s2).all()


NORM_GRADS = [(1, 16), (2, 2048), (7, 2064), (33, 4096), (5, 4112), (3, 8192), (4, 8208), (2, 16384), (2, 16400),
              (1, 32768), (1500, 80), (2000, 1168), (4100, 16), (4096, 1024), (600, 4080), (600, 4096)]


@pytest.mark.parametrize("M,K", NORM_GRADS)
def test_norm_gradient(w8, M, K):
    x, _, w = norm_inputs(M, K, 3 * M + K)
    g = torch.Generator().manual_seed(K)
    dn, dh = torch.randn(M, K, generator=g).to(BF), torch.randn(M, K, generator=g).to(BF)
    for other, wt in [(dh, w), (None, w), (dh, None)]:
        dx, dw = w8.add_rms_norm_backward(*dev(dn, x, wt), eps=1e-5, dh=None if other is None else other.to(DEV))
        want, size, want_dw, dw_size = aref.norm_grad(dn, other, x, wt, 1e-5)
        # reductions: at most 64 values to a lane, 6 exchanges, 16 wavefronts, for both sums; a few operations more
        ref.check(dx, want, 2 * (64 + 22 + 8) * U * size, "dx")
        # rows in a workgroup and the join of the workgroups, each term off by the norm's factor and two roundings
        assert ((dw.cpu().double() - want_dw).abs() <= (M + 64 + 60) * U * dw_size + 1e-30).all()
        again = w8.add_rms_norm_backward(*dev(dn, x, wt), eps=1e-5, dh=None if other is None else other.to(DEV))
        assert same(again[0], dx) and same(again[1], dw)
    got, none = w8.add_rms_norm_backward(*dev(dn, x, w), dweight=False)
    assert none is None and same(got, w8.add_rms_norm_backward(*dev(dn, x, w))[0])


def test_norm_gradient_against_differences(w8):
    """The formula itself: central differences of sum(dn * norm) + sum(dh * h) in 64 bits."""
    M, K, eps = 3, 32, 1e-3
    g = torch.Generator().manual_seed(0)
    h, dn, dh, w = (torch.randn(*s, generator=g).to(BF) for s in ((M, K), (M, K), (M, K), (K,)))

    def loss(h, w):
        return (dn.double() * h / (h.square().mean(1, keepdim=True) + eps).sqrt() * w).sum() + (dh.double() * h).sum()

    dx, dw = w8.add_rms_norm_backward(*dev(dn, h, w), eps=eps, dh=dh.to(DEV))
    step, h64, w64 = 1e-5, h.double(), w.double()
    for at in [(0, 0), (1, 17), (2, 31)]:
        e = torch.zeros_like(h64)
        e[at] = step
        d = (loss(h64 + e, w64) - loss(h64 - e, w64)) / (2 * step)
        assert abs(float(dx[at]) - float(d)) <= 2 ** -8 * abs(float(d)) + 1e-6
        e = torch.zeros_like(w64)
        e[at[1]] = step
        d = (loss(h64, w64 + e) - loss(h64, w64 - e)) / (2 * step)
        assert abs(float(dw[at[1]]) - float(d)) <= 1e-5 * (1 + abs(float(d)))


def test_norm_gradient_in_place_and_empty(w8):
    M, K = 300, 2064
    x, _, w = norm_inputs(M, K, 9)
    dn, dh = torch.randn(M, K).to(BF), torch.randn(M, K).to(BF)
    want = w8.add_rms_norm_backward(*dev(dn, x, w), dh=dh.to(DEV))
    for into in range(3):
        t = list(dev(dn, x, dh))
        got = w8.add_rms_norm_backward(t[0], t[1], w.to(DEV), dh=t[2], dx=t[into])
        assert got[0].data_ptr() == t[into].data_ptr() and same(got[0], want[0]) and same(got[1], want[1])
    e = torch.empty(0, K, dtype=BF, device=DEV)
    q, s, h = w8.add_rms_norm_quantize(e, e, w.to(DEV))
    assert q.shape == (0, K) and s.shape == (0,) and h.shape == (0, K)
    dx, dw = w8.add_rms_norm_backward(e, e, w.to(DEV))
    assert dx.shape == (0, K) and not dw.any()
    # rows of zeros with eps = 0: the residual's gradient passes, the norm adds nothing
    z = torch.zeros(2, K, dtype=BF, device=DEV)
    dx, dw = w8.add_rms_norm_backward(z + 1, z, None, eps=0.0, dh=z + 2)
    assert (dx == 2).all() and not dw.any()


# ---- adapters, forward ----

def adapter_inputs(M, K, N, R, L, kind, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g).to(BF)
    wq, ws = ref.codes_of((torch.randn(N, K, generator=g) * 0.05).to(BF))
    a = (torch.randn(L, R, K, generator=g) / K ** 0.5).to(BF)
    b = (torch.randn(L, N, R, generator=g) * 0.3).to(BF)
    scaling = torch.rand(L, generator=g) * 2 - 0.5      # of either sign
    if kind == "one":
        ids = torch.full((M,), L - 1)
    elif kind == "none":
        ids = torch.full((M,), -1)
    elif kind == "runs":
        ids = torch.arange(M) * L // M
    else:
        ids = torch.randint(-2, L + 2, (M,), generator=g)   # some outside on either side
    bias = torch.randn(N, generator=g).to(BF) if bias else None
    return x, wq, ws, a, b, ids.to(torch.int32), scaling, bias


def check_linear(w8, inputs, what):
    x, wq, ws, a, b, ids, scaling, bias = inputs
    xq, xs = ref.codes_of(x)
    args = dev(wq, ws, a, b, ids, scaling)
    y = w8.linear_adapters(*dev(xq, xs), *args, bias=dev(bias)[0])
    want, slack = aref.linear(xq, xs, wq, ws, a, b, ids, scaling, bias)
    ref.check(y, want, slack, what, rms_steps=1.5)
    # tokens without an adapter: the linear's own bits
    none = ((ids < 0) | (ids >= a.shape[0])).nonzero().flatten().to(DEV)
    plain = w8.linear(*dev(xq, xs, wq, ws, bias))
    assert same(y[none], plain[none]), what
    dyn = w8.linear_adapters_dynamic(x.to(DEV), *args, bias=dev(bias)[0])
    assert same(dyn, y), what
    return y


# few tokens (one and two tiles of them, many groups of channels), the row kernel and the block kernel of the
# first product, the K split, every kind of tile
SHAPES = [(1, 16, 1, 8, 1, "one"), (1, 2048, 2048, 16, 4, "mixed"), (3, 784, 77, 24, 5, "mixed"), (16, 4096, 40, 16, 16, "mixed"),
          (16, 1024, 9001, 40, 3, "mixed"), (17, 1040, 5000, 128, 9, "mixed"), (32, 2048, 16384, 8, 40, "mixed"),
          (16, 20000, 48, 16, 3, "mixed"), (33, 4096, 512, 16, 33, "mixed"), (64, 6144, 256, 64, 7, "mixed"),
          (50, 6144, 264, 8, 2, "runs"), (100, 272, 130, 16, 1, "one"), (256, 512, 300, 72, 4, "runs"),
          (257, 512, 300, 72, 4, "runs"), (300, 1168, 4603, 40, 9, "mixed"), (777, 1168, 603, 128, 70, "mixed"),
          (1000, 256, 1024, 32, 3, "runs"), (2048, 128, 2048, 16, 5, "mixed"), (513, 4096, 513, 48, 2, "none"),
          (260, 20000, 64, 8, 3, "mixed"), (1290, 20000, 64, 8, 3, "mixed"), (1280, 512, 264, 16, 3, "mixed"),
          (160, 512, 300, 120, 4, "mixed"), (161, 512, 300, 120, 4, "mixed"), (4, 1024, 520, 8, 3, "mixed"),
          (1, 1024, 8200, 16, 2, "one"), (2, 1024, 4100, 16, 2, "mixed"), (1, 2048, 300, 32, 3, "one")]


@pytest.mark.parametrize("M,K,N,R,L,kind", SHAPES)
def test_linear_with_adapters(w8, M, K, N, R, L, kind):
    for bias in (True, False):
        check_linear(w8, adapter_inputs(M, K, N, R, L, kind, M + K + N, bias), (M, K, N, R, L, kind))


@pytest.mark.parametrize("M,N,K,R", [(300, 520, 256, 24), (777, 603, 400, 40)])
def test_every_tile_gives_the_same_bits(w8, M, N, K, R):
    x, wq, ws, a, b, ids, scaling, bias = adapter_inputs(M, K, N, R, 6, "mixed", 11)
    xq, xs = ref.codes_of(x)
    args = dev(xq, xs, wq, ws, a, b, ids, scaling, bias)
    ys = [w8.linear_adapters(*args, tile=t) for t in range(w8.num_tiles())]
    want, slack = aref.linear(xq, xs, wq, ws, a, b, ids, scaling, bias)
    ref.check(ys[0], want, slack, "tile 0", rms_steps=1.5)
    for t, y in enumerate(ys):
        assert same(y, ys[0]), t


@pytest.mark.parametrize("M,N,K", [(5, 300, 1024), (16, 5000, 800), (48, 256, 6144), (120, 264, 512), (700, 520, 512)])
def test_other_adapters_do_not_matter(w8, M, N, K):
    """NaNs and infinities in adapters that other tokens have, and what the other tokens are."""
    x, wq, ws, a, b, ids, scaling, bias = adapter_inputs(M, K, N, 16, 4, "mixed", 21)
    xq, xs = ref.codes_of(x)
    y = w8.linear_adapters(*dev(xq, xs, wq, ws, a, b, ids, scaling, bias))
    bad_a, bad_b, bad_s = a.clone(), b.clone(), scaling.clone()
    bad_a[1, 3], bad_b[1, 5], bad_b[1, 7, 2] = float("nan"), float("inf"), float("nan")
    bad_a[2], bad_s[2] = float("-inf"), float("nan")
    got = w8.linear_adapters(*dev(xq, xs, wq, ws, bad_a, bad_b, ids, bad_s, bias))
    keep = ((ids != 1) & (ids != 2)).nonzero().flatten().to(DEV)
    assert same(got[keep], y[keep])
    other = ids.clone()
    other[::3] = (other[::3] + 1) % 4
    got = w8.linear_adapters(*dev(xq, xs, wq, ws, a, b, other, scaling, bias))
    keep = (other == ids).nonzero().flatten().to(DEV)
    assert 0 < len(keep) < M or M < 4
    assert same(got[keep], y[keep])


def test_outputs_workspaces_and_addresses(w8):
    for M, N, K in [(4, 96, 800), (40, 264, 6144), (300, 96, 256)]:
        x, wq, ws, a, b, ids, scaling, bias = dev(*adapter_inputs(M, K, N, 24, 3, "mixed", 31))
        xq, xs = w8.quantize_act(x)
        want = w8.linear_adapters(xq, xs, wq, ws, a, b, ids, scaling, bias)
        room = torch.full((M * N + 9,), 7.0, dtype=BF, device=DEV)
        for off in (0, 1, 8):
            room.fill_(7.0)
            y = room[off:off + M * N].view(M, N)
            assert w8.linear_adapters(xq, xs, wq, ws, a, b, ids, scaling, bias, y=y) is y
            if off % 8 == 0 or M != 40:      # (a K split needs an aligned output)
                assert same(y, want)
            else:
                assert (y.float() - want.float()).abs().max() <= 2 ** -7 * want.float().abs().max()
            assert (room[:off] == 7).all() and (room[off + M * N:] == 7).all()
        need = w8.lib.w8a8_linear_adapters_workspace(M, N, K, 24, 1)
        for fill in (0, 255):
            space = torch.full((need + 32,), fill, dtype=torch.uint8, device=DEV)
            assert same(w8.linear_adapters_dynamic(x, wq, ws, a, b, ids, scaling, bias, workspace=space[:need]), want)
            assert (space[need:] == fill).all()
    e = torch.empty(0, 256, dtype=BF, device=DEV)
    assert w8.linear_adapters_dynamic(e, wq, ws, a, b, ids[:0], scaling, bias).shape == (0, 96)


@pytest.mark.parametrize("M,N,K", [(4, 96, 800), (20, 512, 1024), (40, 264, 6144), (300, 264, 256), (700, 1032, 512)])
def test_scales_and_biases_at_any_address(w8, M, N, K):
    x, wq, ws, a, b, ids, scaling, bias = dev(*adapter_inputs(M, K, N, 24, 3, "mixed", 33))
    xq, xs = w8.quantize_act(x)
    want = w8.linear_adapters(xq, xs, wq, ws, a, b, ids, scaling, bias)

    def moved(t):
        room = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        room[1:] = t
        return room[1:]
    for name in ("xs", "ws", "bias", "ids", "scaling"):
        args = dict(xs=xs, ws=ws, bias=bias, ids=ids, scaling=scaling)
        args[name] = moved(args[name])
        got = w8.linear_adapters(xq, args["xs"], wq, args["ws"], a, b, args["ids"], args["scaling"], args["bias"])
        assert same(got, want), name


# ---- adapters, gradients ----

# every path of dx (few tokens from the codes, tiles whole and in ranges, dy copied or not), rows and blocks of the
# first products, every shape of the matrices' gradients, parts of long lists, adapters without tokens
GRADS = [(1, 16, 1, 8, 1, "one"), (3, 784, 77, 24, 5, "mixed"), (64, 256, 512, 16, 1, "one"), (29, 2592, 2776, 16, 3, "mixed"),
         (64, 2592, 2776, 40, 9, "mixed"), (100, 1024, 5000, 8, 2, "runs"), (257, 512, 300, 72, 4, "runs"),
         (300, 1168, 1203, 40, 9, "mixed"), (777, 528, 603, 128, 70, "mixed"), (1037, 272, 5466, 8, 3, "mixed"),
         (2048, 1024, 1024, 16, 1, "one"), (2100, 512, 2048, 64, 4, "runs"), (3000, 2064, 264, 32, 2, "mixed"),
         (500, 64, 64, 16, 5, "none"), (1300, 1040, 1000, 24, 2, "runs"), (4500, 96, 130, 48, 3, "mixed"),
         (1280, 256, 520, 16, 3, "mixed"), (1290, 304, 523, 8, 300, "mixed")]


def grad_inputs(M, K, N, R, L, kind, seed):
    x, wq, ws, a, b, ids, scaling, _ = adapter_inputs(M, K, N, R, L, kind, seed)
    xq, xs = ref.codes_of(x)
    dy = torch.randn(M, N, generator=torch.Generator().manual_seed(seed + 1)).to(BF)
    return dy, xq, xs, wq, ws, a, b, ids, scaling


@pytest.mark.parametrize("M,K,N,R,L,kind", GRADS)
def test_adapter_gradients(w8, M, K, N, R, L, kind):
    inputs = grad_inputs(M, K, N, R, L, kind, M + K + N)
    got = w8.linear_adapters_backward(*dev(*inputs))
    for g, (want, off), name in zip(got, aref.grads(*inputs), ("dx", "da", "db")):
        assert g.shape == want.shape and g.dtype == BF
        # the operands' roundings add about as much as the output's own, each of an rms of half a step / sqrt(3)
        ref.check(g, want, off, name, rms_steps=2.0)
    again = w8.linear_adapters_backward(*dev(*inputs))
    assert all(same(a, b) for a, b in zip(got, again))
    for asked in [(True, False, False), (False, True, False), (False, False, True), (True, False, True)]:
        some = w8.linear_adapters_backward(*dev(*inputs), *asked)
        for g, s, wanted in zip(got, some, asked):
            assert (s is None) == (not wanted)
            assert s is None or same(s, g)
    for i in range(L):
        if not (inputs[7] == i).any():
            assert not got[1][i].any() and not got[2][i].any()


@pytest.mark.parametrize("M,K,N,R,L,kind", [(1, 512, 520, 8, 1, "one"), (3, 256, 255, 24, 2, "runs"), (22, 256, 255, 8, 7, "runs"),
                                            (16, 512, 264, 128, 2, "mixed"), (128, 256, 264, 16, 3, "mixed")])
def test_few_tokens_gradients_are_rounded_once(w8, M, K, N, R, L, kind):
    """No other error of the adapters' gradients is seen beside their own rounding: fp32 sums, and operands to 2^-17."""
    inputs = grad_inputs(M, K, N, R, L, kind, M + N)
    for got, (want, _) in zip(w8.linear_adapters_backward(*dev(*inputs))[1:], aref.grads(*inputs)[1:]):
        rms = lambda e: float(e.square().mean().sqrt())
        assert rms(got.cpu().double() - want) <= 1.03 * rms(want.to(BF).double() - want)


@pytest.mark.parametrize("R", [8, 24, 40])
@pytest.mark.parametrize("N", [1, 2, 5, 7, 8, 9, 15, 63, 129])
def test_gradients_of_few_channels(w8, N, R):
    for M in (31, 70, 600):
        inputs = grad_inputs(M, 48, N, R, 2, "mixed", M + N + R)
        got = w8.linear_adapters_backward(*dev(*inputs))
        for g, (want, off), name in zip(got, aref.grads(*inputs), ("dx", "da", "db")):
            ref.check(g, want, off, name, rms_steps=2.5)   # (fewer elements than elsewhere)


@pytest.mark.parametrize("M,R", [(1, 8), (40, 8), (289, 16), (300, 32), (700, 64)])
def test_infinities_in_an_outputs_gradient(w8, M, R):
    """They stay in their channel and adapter, and are no NaN."""
    N, K = 136, 64
    dy, xq, xs, wq, ws, a, b, ids, scaling = grad_inputs(M, K, N, R, 2, "runs", M)
    plain = w8.linear_adapters_backward(*dev(dy, xq, xs, wq, ws, a, b, ids, scaling))[2]
    bad = dy.clone()
    bad[M - 1, 3], bad[0, 77] = float("inf"), float("-inf")   # the last of a list that fills no step, and a first one
    got = w8.linear_adapters_backward(*dev(bad, xq, xs, wq, ws, a, b, ids, scaling))[2].cpu()
    hit = torch.zeros(2, N, dtype=torch.bool)
    hit[ids[M - 1], 3] = hit[ids[0], 77] = True
    assert torch.isinf(got[hit]).all()
    assert same(got[~hit], plain.cpu()[~hit])


def test_tokens_without_adapters_have_the_linears_gradient(w8):
    for M, N, K in [(40, 2776, 2592), (300, 520, 256), (700, 2048, 512)]:
        inputs = dev(*grad_inputs(M, K, N, 16, 3, "none", 3))
        dx, da, db = w8.linear_adapters_backward(*inputs)
        want = w8.linear_backward(*inputs[:5], dw=False, dbias=False)[0]
        # (the same sums; the tiles of a large product may be others, and with them the sums' order)
        ref.check(dx, want.cpu().double(), 2 * N * U * float(want.abs().max()) * 4, "dx", rms_steps=1.5)
        assert not da.any() and not db.any()


def test_adapter_gradients_against_differences(w8):
    """The formulas themselves: the gradients of sum(dy * y) in 64 bits by central differences."""
    M, K, N, R, L = 5, 32, 24, 8, 2
    inputs = grad_inputs(M, K, N, R, L, "mixed", 77)
    dy, xq, xs, wq, ws, a, b, ids, scaling = inputs
    x0 = xq.double() * xs.double()[:, None]
    w = wq.double() * ws.double()[:, None]

    def loss(x, a, b):
        y = x @ w.T
        for i in range(L):
            at = ids == i
            y[at] += scaling[i].double() * (x[at] @ a[i].T) @ b[i].T
        return (y * dy.double()).sum()

    got = w8.linear_adapters_backward(*dev(*inputs))
    args = [x0, a.double(), b.double()]
    offs = [o for _, o in aref.grads(*inputs)]
    g = torch.Generator().manual_seed(1)
    for k, (t, grad, off) in enumerate(zip(args, got, offs)):
        for _ in range(6):
            at = tuple(int(torch.randint(0, n, (1,), generator=g)) for n in t.shape)
            e = torch.zeros_like(t)
            e[at] = 1e-3
            up_, down_ = [list(args), list(args)]
            up_[k], down_[k] = t + e, t - e
            d = float((loss(*up_) - loss(*down_)) / 2e-3)
            assert abs(float(grad[at]) - d) <= float(off[at]) + 2 ** -8 * abs(d) + 1e-9, (k, at)


@pytest.mark.parametrize("M,N,K", [(40, 96, 64), (64, 2776, 2592), (700, 520, 512)])
def test_other_adapters_do_not_matter_to_gradients(w8, M, N, K):
    dy, xq, xs, wq, ws, a, b, ids, scaling = grad_inputs(M, K, N, 16, 4, "mixed", 5)
    got = w8.linear_adapters_backward(*dev(dy, xq, xs, wq, ws, a, b, ids, scaling))
    bad_a, bad_b, bad_s = a.clone(), b.clone(), scaling.clone()
    bad_a[1, 3], bad_b[1, 5], bad_s[1] = float("nan"), float("inf"), float("nan")
    bad = w8.linear_adapters_backward(*dev(dy, xq, xs, wq, ws, bad_a, bad_b, ids, bad_s))
    keep = (ids != 1).nonzero().flatten().to(DEV)
    assert same(bad[0][keep], got[0][keep])
    others = [0, 2, 3]
    assert same(bad[1][others], got[1][others]) and same(bad[2][others], got[2][others])
    # a NaN token is its own adapter's trouble alone
    xs2 = xs.clone()
    m = int((ids == 2).nonzero()[0])
    xs2[m] = float("nan")
    bad = w8.linear_adapters_backward(*dev(dy, xq, xs2, wq, ws, a, b, ids, scaling))
    others = [0, 1, 3]
    assert same(bad[0], got[0]) and same(bad[1][others], got[1][others]) and same(bad[2][others], got[2][others])


def test_gradient_workspaces_and_addresses(w8):
    for M, N, K in [(50, 2776, 2592), (300, 520, 256), (600, 77, 128)]:
        dy, xq, xs, wq, ws, a, b, ids, scaling = dev(*grad_inputs(M, K, N, 24, 3, "mixed", 8))
        want = w8.linear_adapters_backward(dy, xq, xs, wq, ws, a, b, ids, scaling)
        need = w8.lib.w8a8_linear_adapters_backward_workspace(M, N, K, 24, 3, 1, 1, 1)
        for fill in (0, 255):
            space = torch.full((need + 32,), fill, dtype=torch.uint8, device=DEV)
            got = w8.linear_adapters_backward(dy, xq, xs, wq, ws, a, b, ids, scaling, workspace=space[:need])
            assert all(same(x, y) for x, y in zip(got, want)) and (space[need:] == fill).all()
        # dy at an odd address
        room = torch.empty(M * N + 1, dtype=BF, device=DEV)
        odd = room[1:].view(M, N)
        odd.copy_(dy)
        got = w8.linear_adapters_backward(odd, xq, xs, wq, ws, a, b, ids, scaling)
        assert same(got[1], want[1]) and same(got[2], want[2])
        ref.check(got[0], want[0].cpu().double(), 2 * N * U * float(want[0].abs().max()) * 4, "dx", rms_steps=1.5)
    e = torch.empty(0, 77, dtype=BF, device=DEV)
    dx, da, db = w8.linear_adapters_backward(e, xq[:0], xs[:0], wq, ws, a, b, ids[:0], scaling)
    assert dx.shape == (0, 128) and not da.any() and not db.any() and da.shape == a.shape and db.shape == b.shape


@pytest.mark.parametrize("M,K,N,R,L,kind", SHAPES + GRADS)
def test_the_adapters_share_alone(w8, M, K, N, R, L, kind):
    """A weight of scale zero leaves the adapters' products and their rounding."""
    x, wq, ws, a, b, ids, scaling, _ = adapter_inputs(M, K, N, R, L, kind, M + K + N + R)
    xq, xs = ref.codes_of(x)
    ws = torch.zeros_like(ws)
    y = w8.linear_adapters(*dev(xq, xs, wq, ws, a, b, ids, scaling))
    ref.check(y, *aref.linear(xq, xs, wq, ws, a, b, ids, scaling, None), "y", rms_steps=2.0)
    dy = torch.randn(M, N, generator=torch.Generator().manual_seed(M)).to(BF)
    dx = w8.linear_adapters_backward(*dev(dy, xq, xs, wq, ws, a, b, ids, scaling), da=False, db=False)[0]
    ref.check(dx, *aref.grads(dy, xq, xs, wq, ws, a, b, ids, scaling)[0], "dx", rms_steps=2.0)


# sizes whose products take each of the larger tiles, whole and in ranges
LARGE = [(3000, 4096, 600, 16, 3, "mixed"), (4096, 2048, 264, 64, 2, "runs"), (2000, 2976, 1024, 40, 2, "runs"),
         (777, 2976, 8192, 16, 4, "mixed"), (1500, 2064, 1024, 8, 3, "mixed"), (1500, 1024, 8192, 64, 5, "runs"),
         (300, 4096, 600, 24, 2, "mixed"), (520, 1024, 8192, 16, 9, "mixed"), (2000, 1024, 256, 16, 1, "one"),
         (520, 256, 4096, 128, 3, "mixed"), (1037, 512, 8192, 16, 2, "runs"), (8192, 512, 1536, 16, 20, "mixed")]


@pytest.mark.parametrize("M,K,N,R,L,kind", LARGE)
def test_larger_products(w8, M, K, N, R, L, kind):
    for scale in (1.0, 0.0):      # (0: the adapters' share alone)
        x, wq, ws, a, b, ids, scaling, bias = dev(*adapter_inputs(M, K, N, R, L, kind, M + K + N))
        ws = ws * scale
        xq, xs = w8.quantize_act(x)
        y = w8.linear_adapters(xq, xs, wq, ws, a, b, ids, scaling, bias if scale else None)
        want, slack = aref.linear(xq, xs, wq, ws, a, b, ids, scaling, bias if scale else None)
        ref.check(y, want, slack.cpu(), "y", rms_steps=2.0)
        dy = torch.randn(M, N, device=DEV).to(BF)
        got = w8.linear_adapters_backward(dy, xq, xs, wq, ws, a, b, ids, scaling)
        for g, (want, off), name in zip(got, aref.grads(dy, xq, xs, wq, ws, a, b, ids, scaling), ("dx", "da", "db")):
            ref.check(g, want, off.cpu(), name, rms_steps=2.0)
