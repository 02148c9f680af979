"""GPU checks of the operators around the linear against plain 64-bit forms:
the few-token forms (bit-identical to quantize + linear), the gated product,
the backward passes, and the norm and rotation of queries and keys.

Bounds.  bf16 rounding is at most 2^-8 of the value.  A scaled product value is
an exact integer through three or four fp32 roundings (2^-24 each) of a value at
most |acc sx sw| + |b|; activations are within 3e-5.  In a gradient product one
operand is rounded to bf16 once (2^-8 of each term) and the fp32 sum of n terms
is within n 2^-24 of the terms' magnitudes."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    import w8a8_int8_quantized_token_amd as pkg
    return pkg


def gen(seed):
    return torch.Generator().manual_seed(seed)


def weights(rows, K, g, bias):
    wq, ws = ref.codes_of((torch.randn(rows, K, generator=g) * 0.05).to(BF))
    b = (torch.randn(rows, generator=g) * 0.2).to(BF) if bias else None
    return wq, ws, b


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def bits(t):
    return t.detach().cpu().view(torch.int16)


# ---- few tokens ----

FEW = [(1, 128, 16), (1, 1, 16), (2, 33, 48), (3, 17, 4112), (4, 200, 272), (5, 129, 1040), (8, 64, 64), (9, 100, 2064),
       (16, 257, 1024), (17, 48, 528), (31, 1000, 336), (32, 96, 4096), (32, 40, 8208), (1, 2048, 12288),
       (16, 48, 16400), (1, 24, 133136), (33, 72, 160), (40, 8, 8192), (100, 264, 2048)]


@pytest.mark.parametrize("M,N,K", FEW)
@pytest.mark.parametrize("gelu,bias", [(False, True), (True, False)])
def test_linear_dynamic_has_the_bits_of_quantize_and_linear(w8, M, N, K, gelu, bias):
    g = gen(M * 7 + N)
    wq, ws, b = dev(*weights(N, K, g, bias))
    x = torch.randn(M, K, generator=g)
    x[M // 2] = 0.0 if M > 1 else x[0]      # a row without a largest value
    x = x.to(BF).to(DEV)
    y = w8.linear_dynamic(x, wq, ws, b, gelu=gelu)
    want = w8.linear(*w8.quantize_act(x), wq, ws, b, gelu=gelu)
    torch.cuda.synchronize()
    assert torch.equal(bits(y), bits(want))


@pytest.mark.parametrize("M,N,K", FEW)
@pytest.mark.parametrize("kind,bias", [("silu", True), ("gelu", False)])
def test_gated_dynamic_has_the_bits_of_quantize_and_gated(w8, M, N, K, kind, bias):
    g = gen(M * 5 + N)
    wq, ws, b = dev(*weights(2 * N, K, g, bias))
    x = torch.randn(M, K, generator=g).to(BF).to(DEV)
    y = w8.gated_linear_dynamic(x, wq, ws, b, act=kind)
    want = w8.gated_linear(*w8.quantize_act(x), wq, ws, b, act=kind)
    torch.cuda.synchronize()
    assert torch.equal(bits(y), bits(want))


def test_few_tokens_of_tiny_and_huge_values(w8):
    # scales below the smallest normal quotient's range and near the largest
    g = gen(3)
    wq, ws, b = dev(*weights(64, 128, g, True))
    x = torch.randn(4, 128, generator=g)
    x[0] *= 2.0 ** -120
    x[1] *= 2.0 ** 100
    x[2] = 0
    x = x.to(BF).to(DEV)
    assert torch.equal(bits(w8.linear_dynamic(x, wq, ws, b)), bits(w8.linear(*w8.quantize_act(x), wq, ws, b)))


# ---- gated product ----

GATED = [(1, 1, 16), (7, 5, 48), (64, 96, 256), (130, 97, 272), (257, 120, 1040), (300, 1001, 512), (513, 384, 4096),
         (1024, 520, 144)]


@pytest.mark.parametrize("M,N,K", GATED)
@pytest.mark.parametrize("kind,bias", [("silu", True), ("gelu", False)])
def test_gated_linear(w8, M, N, K, kind, bias):
    g = gen(M + N)
    wq, ws, b = weights(2 * N, K, g, bias)
    xq, xs = ref.codes_of(torch.randn(M, K, generator=g).to(BF))
    y = w8.gated_linear(*dev(xq, xs, wq, ws, b), act=kind)
    want = ref.gated(xq, xs, wq, ws, b, kind)
    z = ref.product(xq, xs, wq, ws, b)
    mag = z.abs() + (0 if b is None else b.to(ref.F64).abs())     # what the fp32 roundings are relative to
    gm, um = mag.chunk(2, 1)
    slack = (3e-5 + 8 * 2.0 ** -24) * 1.2 * gm * um
    ref.check(y, want, slack, "y")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_every_tile_gives_the_same_gated_bits(w8, kind):
    M, N, K = 777, 1032, 400
    g = gen(11)
    args = dev(*ref.codes_of(torch.randn(M, K, generator=g).to(BF)), *weights(2 * N, K, g, True))
    outs = [bits(w8.gated_linear(*args, act=kind, tile=t)) for t in range(w8.num_tiles())]
    for t, o in enumerate(outs):
        assert torch.equal(o, outs[0]), t


def test_gated_with_a_tail_plan(w8):
    # sizes where the main tiles come out as whole waves and the rest of the
    # channels goes to the second launch
    M, K = 4096, 64
    N = 256 * 9 + 40
    g = gen(12)
    args = dev(*ref.codes_of(torch.randn(M, K, generator=g).to(BF)), *weights(2 * N, K, g, True))
    outs = [bits(w8.gated_linear(*args, tile=t)) for t in (0, 1, 2, 4)]
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_gated_extremes(w8):
    # far negative and positive gates: no NaN from an overflowing exponential
    wq, ws, b = weights(16, 16, gen(1), False)
    b = torch.cat([torch.linspace(-3e4, 3e4, 8), torch.ones(8)]).to(BF)
    xq, xs = torch.zeros(3, 16, dtype=torch.int8), torch.zeros(3)
    for kind in ("silu", "gelu"):
        y = w8.gated_linear(*dev(xq, xs, wq, ws, b), act=kind)
        ref.check(y, ref.gated(xq, xs, wq, ws, b, kind), torch.tensor(1e-30), kind)


# ---- backward ----

BACK = [(1, 1, 16), (8, 8, 32), (9, 7, 48), (65, 33, 272), (130, 96, 128), (300, 257, 528), (777, 1001, 400),
        (64, 2048, 256), (2049, 64, 144), (3, 1601, 2000), (40, 1999, 1568)]


def grad_slack(mag, n):
    return (ref.BF16_HALF_STEP + (n + 40) * 2.0 ** -24) * mag


@pytest.mark.parametrize("M,N,K", BACK)
def test_linear_backward(w8, M, N, K):
    g = gen(M + 3 * N)
    wq, ws, _ = weights(N, K, g, False)
    xq, xs = ref.codes_of(torch.randn(M, K, generator=g).to(BF))
    dy = torch.randn(M, N, generator=g).to(BF)
    (dx, dxm), (dw, dwm), (db, dbm) = ref.product_grads(dy.to(ref.F64), xq, xs, wq, ws)
    got = w8.linear_backward(*dev(dy, xq, xs, wq, ws))
    ref.check(got[0], dx, grad_slack(dxm, N), "dx")
    ref.check(got[1], dw, grad_slack(dwm, M), "dw")
    ref.check(got[2], db, (M + 2) * 2.0 ** -24 * dbm, "dbias")
    # each output alone, the same bits
    for i, name in enumerate(("dx", "dw", "dbias")):
        flags = {n: n == name for n in ("dx", "dw", "dbias")}
        alone = w8.linear_backward(*dev(dy, xq, xs, wq, ws), **flags)
        assert [a is not None for a in alone] == [n == name for n in ("dx", "dw", "dbias")]
        assert torch.equal(bits(alone[i]), bits(got[i])), name


# shapes of dx whose product takes each of its tiles whole or in ranges of the
# sum, on both sides of copying dy for the sake of its rows' alignment, and few
# tokens of a large weight
TILES = [(10079, 1026, 1216), (3872, 201, 3488), (4925, 278, 2272), (987, 520, 6544), (4500, 8, 144),
         (397, 1021, 5920), (186, 141, 8336), (69, 135, 8720),
         (434, 10056, 9104), (2088, 9573, 2208), (6308, 12097, 160), (66, 11925, 6032), (84, 8175, 2528),
         (67, 4974, 7904), (1, 2197, 2624), (2545, 2170, 16), (1, 1296, 16), (300, 2056, 512), (300, 2056, 496),
         (1, 2501, 2624), (15, 1200, 5008), (16, 6001, 1008), (17, 9000, 752), (32, 12504, 496), (33, 3333, 1904),
         (48, 23001, 272), (64, 777, 8208), (65, 777, 8208)]


@pytest.mark.parametrize("M,N,K", TILES)
def test_input_gradient_on_every_tile(w8, M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M + N)
    wq = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    ws = torch.rand(N, generator=g, device=DEV) * 0.02 + 1e-3
    dy = torch.randn(M, N, generator=g, device=DEV).to(BF)
    w = wq.to(ref.F64) * ws.to(ref.F64)[:, None]
    want = dy.to(ref.F64) @ w
    mag = dy.to(ref.F64).abs() @ w.abs()
    got = w8.linear_backward(dy, None, None, wq, ws, dw=False, dbias=False)[0]
    ref.check(got, want.cpu(), grad_slack(mag.cpu(), N), "dx")
    assert torch.equal(bits(w8.linear_backward(dy, None, None, wq, ws, dw=False, dbias=False)[0]), bits(got))


def test_linear_backward_of_an_unaligned_dy(w8):
    M, N, K = 40, 64, 96
    g = gen(5)
    wq, ws, xq, xs = dev(*weights(N, K, g, False)[:2], *ref.codes_of(torch.randn(M, K, generator=g).to(BF)))
    dy = torch.randn(M, N, generator=g).to(BF)
    odd = torch.empty(M * N + 1, dtype=BF, device=DEV)[1:].view(M, N)
    odd.copy_(dy)
    for a, b in zip(w8.linear_backward(odd, xq, xs, wq, ws), w8.linear_backward(dy.to(DEV), xq, xs, wq, ws)):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("M,N,K", BACK)
@pytest.mark.parametrize("kind,bias", [("silu", True), ("gelu", False)])
def test_gated_linear_backward(w8, M, N, K, kind, bias):
    g = gen(M + 5 * N)
    wq, ws, b = weights(2 * N, K, g, bias)
    xq, xs = ref.codes_of(torch.randn(M, K, generator=g).to(BF))
    dy = torch.randn(M, N, generator=g).to(BF)
    d = ref.gated_d(dy, xq, xs, wq, ws, b, kind)
    # errors of g and u move d: |act'|, |act''| <= 1.2 for both activations
    z = ref.product(xq, xs, wq, ws, b)
    mag = z.abs() + (0 if b is None else b.to(ref.F64).abs())
    gm, um = mag.chunk(2, 1)
    dm = dy.to(ref.F64).abs()
    d_err = torch.cat([dm * (1.3 * um * (4e-5 + 10 * 2.0 ** -24 * (1 + gm))), dm * (gm + 1) * 5e-5], 1)
    (dx, dxm), (dw, dwm), (db, dbm) = ref.product_grads(d, xq, xs, wq, ws)
    (_, ex), (_, ew), (_, eb) = ref.product_grads(d_err, xq, xs, wq, ws)
    args = dev(dy, xq, xs, wq, ws, b)
    got = w8.gated_linear_backward(*args, act=kind)
    ref.check(got[0], dx, grad_slack(dxm, 2 * N) + 2 * ex, "dx")
    ref.check(got[1], dw, grad_slack(dwm, M) + 2 * ew, "dw")
    ref.check(got[2], db, (M + 2) * 2.0 ** -24 * dbm + eb, "dbias")
    for i, name in enumerate(("dx", "dw", "dbias")):
        flags = {n: n == name for n in ("dx", "dw", "dbias")}
        alone = w8.gated_linear_backward(*args, act=kind, **flags)
        assert torch.equal(bits(alone[i]), bits(got[i])), name


def test_gradients_of_no_tokens_are_zeros(w8):
    N, K = 24, 64
    wq, ws, _ = dev(*weights(2 * N, K, gen(1), False))
    e = [torch.empty(0, N, dtype=BF, device=DEV), torch.empty(0, K, dtype=torch.int8, device=DEV),
         torch.empty(0, device=DEV)]
    for r in (w8.linear_backward(*e, wq[:N].contiguous(), ws[:N].contiguous()), w8.gated_linear_backward(*e, wq, ws)):
        assert r[0].shape == (0, K) and not r[1].any() and not r[2].any()
    assert w8.linear_dynamic(torch.empty(0, K, dtype=BF, device=DEV), wq, ws).shape == (0, 2 * N)
    assert w8.gated_linear_dynamic(torch.empty(0, K, dtype=BF, device=DEV), wq, ws).shape == (0, N)


# ---- norm and rotation ----

ROPE = [  # M, P, Hq, Hk, D, rot
    (1, 7, 1, 1, 16, 16), (3, 3, 2, 1, 32, 16), (5, 2, 4, 2, 48, 32), (17, 40, 3, 3, 64, 64), (9, 100, 10, 2, 80, 80),
    (33, 33, 5, 1, 96, 32), (64, 16, 32, 8, 128, 128), (7, 9, 2, 2, 160, 160), (12, 5, 3, 1, 256, 64),
    (4, 4, 2, 1, 512, 512), (2, 2, 1, 1, 1024, 256), (700, 512, 6, 2, 128, 0)]


def rope_inputs(M, P, Hq, Hk, D, rot, seed, packed=True):
    g = gen(seed)
    qkv = (torch.randn(M, (Hq + 2 * Hk) * D, generator=g) * 3).to(BF).to(DEV)
    q, k = qkv[:, :Hq * D].view(M, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(M, Hk, D)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(BF).to(DEV) for _ in range(2)]
    ang = torch.rand(P, rot // 2, generator=g) * 6.3
    return q, k, w, ang.cos().to(DEV), ang.sin().to(DEV), g


def rows_of(t, M, P, positions=None):
    at = torch.arange(M) % P if positions is None else positions.long().cpu()
    return t.cpu()[at.clamp(0, P - 1)]


@pytest.mark.parametrize("M,P,Hq,Hk,D,rot", ROPE)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("mode", ["plain", "positions", "no weight"])
def test_qk_norm_rope_and_its_gradient(w8, M, P, Hq, Hk, D, rot, interleaved, mode):
    q, k, (qw, kw), cos, sin, g = rope_inputs(M, P, Hq, Hk, D, rot, M * 3 + D)
    if mode == "no weight":
        qw = kw = None
    pos = torch.randint(0, P, (M,), generator=g, dtype=torch.int32) if mode == "positions" else None
    c, s = rows_of(cos, M, P, pos), rows_of(sin, M, P, pos)
    dpos = None if pos is None else pos.to(DEV)
    eps = 1e-5
    got = w8.qk_norm_rope(q, k, qw, kw, cos, sin, dpos, eps=eps, interleaved=interleaved)
    dq = torch.randn(M, Hq, D, generator=g).to(BF)
    dk = torch.randn(M, Hk, D, generator=g).to(BF)
    back = w8.qk_norm_rope_backward(*dev(dq, dk), q, k, qw, kw, cos, sin, dpos, eps=eps, interleaved=interleaved)
    for i, (x, w, dy) in enumerate(((q, qw, dq), (k, kw, dk))):
        wc = None if w is None else w.cpu()
        y = ref.norm_rope(x.cpu(), wc, c, s, eps, interleaved)
        # a rotated value is a sum of two terms, each within about D + 8 fp32 steps
        top = y.abs().amax(-1, keepdim=True)
        ref.check(got[i], y, (D + 16) * 2.0 ** -24 * 2 * top, f"out {i}")
        dx, dw, dwm = ref.norm_rope_grad(dy, x.cpu(), wc, c, s, eps, interleaved)
        ref.check(back[i], dx, (2 * D + 32) * 2.0 ** -24 * 4 * dx.abs().amax(-1, keepdim=True) + 1e-6 *
                  dx.abs().amax(), f"grad {i}")
        n = M * x.shape[1]
        err = (back[2 + i].cpu().to(ref.F64) - dw).abs()
        assert bool((err <= (n + D + 32) * 2.0 ** -24 * dwm + 1e-30).all()), float(err.max())


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_in_place_and_padding_rows(w8, interleaved):
    M, P, Hq, Hk, D = 37, 50, 6, 2, 128
    q, k, (qw, kw), cos, sin, g = rope_inputs(M, P, Hq, Hk, D, 64, 8)
    pos = torch.randint(0, P, (M,), generator=g, dtype=torch.int32)
    pos[3], pos[20], pos[36] = -1, P, 2 ** 31 - 1
    pos = pos.to(DEV)
    want = w8.qk_norm_rope(q, k, qw, kw, cos, sin, pos, interleaved=interleaved)
    for r in (3, 20, 36):
        assert not want[0][r].any() and not want[1][r].any()
    dq, dk = torch.randn_like(want[0]), torch.randn_like(want[1])
    g1 = w8.qk_norm_rope_backward(dq, dk, q, k, qw, kw, cos, sin, pos, interleaved=interleaved)
    keep = [r for r in range(M) if r not in (3, 20, 36)]
    g2 = w8.qk_norm_rope_backward(dq[keep], dk[keep], q[keep], k[keep], qw, kw, cos, sin, pos[keep],
                                  interleaved=interleaved)
    for i in range(2):
        assert not g1[i][[3, 20, 36]].any()
        assert torch.equal(bits(g1[i][keep]), bits(g2[i]))
        assert torch.allclose(g1[2 + i], g2[2 + i], rtol=1e-4, atol=1e-4 * float(g2[2 + i].abs().max()))
    v = q.storage_offset()
    assert v == 0
    w8.qk_norm_rope(q, k, qw, kw, cos, sin, pos, interleaved=interleaved, q_out=q, k_out=k)
    assert torch.equal(bits(q.contiguous()), bits(want[0])) and torch.equal(bits(k.contiguous()), bits(want[1]))


def test_rope_strides_and_shared_heads(w8):
    # heads first in memory, and one key head given to all by a zero stride
    M, P, H, D = 21, 21, 4, 64
    q, k, (qw, kw), cos, sin, g = rope_inputs(M, P, H, 1, D, D, 4)
    qt = q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    ke = k.expand(M, H, D)
    a = w8.qk_norm_rope(q, k, qw, kw, cos, sin)
    b = w8.qk_norm_rope(qt, ke, qw, kw, cos, sin)
    assert torch.equal(bits(a[0]), bits(b[0]))
    for h in range(H):
        assert torch.equal(bits(a[1][:, 0].contiguous()), bits(b[1][:, h].contiguous()))
    with pytest.raises(ValueError):
        w8.qk_norm_rope(q, ke, qw, kw, cos, sin, k_out=ke)      # outputs may not overlap


def test_rope_of_zero_rows_and_zero_vectors(w8):
    q, k, (qw, kw), cos, sin, _ = rope_inputs(4, 4, 2, 1, 64, 64, 2)
    q.zero_()
    a = w8.qk_norm_rope(q, k, qw, kw, cos, sin)
    assert not a[0].any()
    b = w8.qk_norm_rope_backward(torch.ones_like(a[0]), torch.ones_like(a[1]), q, k, qw, kw, cos, sin)
    assert all(torch.isfinite(t).all() for t in b)
    e = w8.qk_norm_rope(q[:0], k[:0], qw, kw, cos, sin)
    assert e[0].shape == (0, 2, 64)
    b = w8.qk_norm_rope_backward(e[0], e[1], q[:0], k[:0], qw, kw, cos, sin)
    assert not b[2].any() and not b[3].any()


def test_rope_of_queries_or_keys_alone(w8):
    q, k, (qw, kw), cos, sin, _ = rope_inputs(9, 9, 4, 2, 64, 64, 6)
    none = q[:, :0]
    both = w8.qk_norm_rope(q, k, qw, kw, cos, sin)
    one = w8.qk_norm_rope(q, none, qw, None, cos, sin)
    other = w8.qk_norm_rope(none, k, None, kw, cos, sin)
    assert torch.equal(bits(one[0]), bits(both[0])) and one[1].shape == (9, 0, 64)
    assert torch.equal(bits(other[1]), bits(both[1]))
    g = w8.qk_norm_rope_backward(q, k, q, k, qw, kw, cos, sin)
    g1 = w8.qk_norm_rope_backward(q, none, q, none, qw, None, cos, sin)
    g2 = w8.qk_norm_rope_backward(none, k, none, k, None, kw, cos, sin)
    assert torch.equal(bits(g1[0]), bits(g[0])) and torch.equal(bits(g2[1]), bits(g[1]))
    assert not g1[3].any() and not g2[2].any()


@pytest.mark.parametrize("M,N,K", [(64, 256, 4096), (40, 64, 128), (300, 136, 64), (5, 24, 64)])
def test_outputs_at_odd_addresses(w8, M, N, K):
    g = gen(M)
    wq, ws, b = dev(*weights(2 * N, K, g, True))
    x = torch.randn(M, K, generator=g).to(BF).to(DEV)
    for f, n in ((w8.linear_dynamic, 2 * N), (w8.gated_linear_dynamic, N)):
        room = torch.empty(M * n + 1, dtype=BF, device=DEV)
        assert torch.equal(bits(f(x, wq, ws, b, y=room[1:].view(M, n))), bits(f(x, wq, ws, b)))


@pytest.mark.parametrize("M,N,K", [(10079, 1026, 1216), (3872, 201, 3488), (4925, 278, 2272), (987, 520, 6544),
                                   (4500, 8, 144), (434, 10056, 9104), (66, 11925, 6032)])
def test_input_gradient_at_an_odd_address(w8, M, N, K):
    """On large tiles, nothing written around it (ranges of the sum are not
    joined at an odd address: the sums run in another order)."""
    g = torch.Generator(device=DEV).manual_seed(M)
    wq = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    ws = torch.rand(N, generator=g, device=DEV) * 0.02 + 1e-3
    dy = torch.randn(M, N, generator=g, device=DEV).to(BF)
    room = torch.full((M * K + 9,), -7.0, dtype=BF, device=DEV)
    need = w8.lib.w8a8_linear_backward_workspace(M, N, K, 1, 0, 0)
    space = torch.empty(need, dtype=torch.uint8, device=DEV)
    status = w8.lib.w8a8_linear_backward(dy.data_ptr(), None, None, wq.data_ptr(), ws.data_ptr(),
                                         room[1:].data_ptr(), None, None, M, N, K, space.data_ptr(), need,
                                         torch.cuda.current_stream().cuda_stream)
    assert status == 0
    got = room[1:1 + M * K].view(M, K)
    w = wq.to(ref.F64) * ws.to(ref.F64)[:, None]
    mag = dy.to(ref.F64).abs() @ w.abs()
    ref.check(got, (dy.to(ref.F64) @ w).cpu(), grad_slack(mag.cpu(), N), "dx")
    assert float(room[0]) == -7.0 and bool((room[1 + M * K:] == -7.0).all())
