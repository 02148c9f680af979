"""The operators around the linear as a program uses them: the modules and
their gradients, all of them in one block, captured graphs, other streams,
shared workspaces, and sizes whose offsets pass 32 bits."""
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


def bits(t):
    return t.detach().contiguous().cpu().view(torch.int16)


def same(a, b):
    return torch.equal(bits(a), bits(b))


def rel(got, want):
    got, want = got.detach().cpu().double(), want.detach().cpu().double()
    return float((got - want).norm() / want.norm())


def linears(w8, seed, *shapes, bias=True):
    torch.manual_seed(seed)
    return [torch.nn.Linear(k, n, bias=bias, device=DEV, dtype=BF) for n, k in shapes]


# ---- modules ----

@pytest.mark.parametrize("tokens", [(1,), (5,), (2, 37), (3, 130)])
def test_linear_module_is_quantize_and_linear_and_differentiable(w8, tokens):
    lin, = linears(w8, 1, (96, 64))
    m = w8.W8A8Linear.from_linear(lin)
    x = torch.randn(*tokens, 64, device=DEV).to(BF)
    want = w8.linear(*w8.quantize_act(x.reshape(-1, 64)), m.wq, m.w_scale, m.bias)
    assert same(m(x).reshape(-1, 96), want) and not m(x).requires_grad
    xg = x.clone().requires_grad_()
    y = m(xg)
    assert same(y.reshape(-1, 96), want)
    dy = torch.randn_like(y)
    y.backward(dy)
    dx = w8.linear_backward(dy.reshape(-1, 96), None, None, m.wq, m.w_scale, dw=False, dbias=False)[0]
    assert same(xg.grad.reshape(-1, 64), dx)
    w = m.wq.double() * m.w_scale.double()[:, None]
    assert rel(xg.grad, dy.double() @ w) < 2 ** -8
    with torch.no_grad():
        assert not m(xg).requires_grad
    # the gradient of a broadcast sum: dy with zero strides
    xg.grad = None
    m(xg).sum().backward()
    assert rel(xg.grad, torch.ones_like(dy).double() @ w) < 2 ** -8


def test_gated_module_and_its_gradient(w8):
    K, H, M = 96, 160, 70
    gate, up, down = linears(w8, 2, (H, K), (H, K), (K, H))
    for act in ("silu", "gelu"):
        m = w8.W8A8GatedMLP.from_linears(gate, up, down, act)
        x = torch.randn(2, M // 2, K, device=DEV).to(BF)
        h = w8.gated_linear(*w8.quantize_act(x.reshape(M, K)), m.wq, m.w_scale, m.bias, act=act)
        want = m.down(h)
        assert same(m(x).reshape(M, K), want)
        xg = x.clone().requires_grad_()
        y = m(xg)
        assert same(y.reshape(M, K), want)
        dy = torch.randn_like(y)
        y.backward(dy)
        dh = w8.linear_backward(dy.reshape(M, K), None, None, m.down.wq, m.down.w_scale, dw=False, dbias=False)[0]
        xq, xs = w8.quantize_act(x.reshape(M, K))
        dx = w8.gated_linear_backward(dh, xq, xs, m.wq, m.w_scale, m.bias, act=act, dw=False, dbias=False)[0]
        assert same(xg.grad.reshape(M, K), dx)
    with pytest.raises(ValueError):
        w8.W8A8GatedMLP.from_linears(gate, down, down)
    with pytest.raises(ValueError):
        w8.W8A8GatedMLP.from_linears(gate, up, down, "relu")
    with pytest.raises(ValueError):
        w8.W8A8GatedMLP.from_linears(gate, torch.nn.Linear(K, H, bias=False, device=DEV, dtype=BF), down)


@pytest.mark.parametrize("interleaved", [False, True])
def test_qkv_module_and_its_gradient(w8, interleaved):
    K, Hq, Hk, D, B, S = 64, 4, 2, 32, 2, 19
    proj, = linears(w8, 3, ((Hq + 2 * Hk) * D, K))
    qw, kw = (1 + 0.2 * torch.randn(D, device=DEV)).to(BF), (1 + 0.2 * torch.randn(D, device=DEV)).to(BF)
    m = w8.W8A8QKV(w8.W8A8Linear.from_linear(proj), Hq, Hk, qw, kw, interleaved=interleaved)
    a = torch.rand(S, D // 2, device=DEV) * 6
    x = torch.randn(B, S, K, device=DEV).to(BF)
    with torch.no_grad():
        q, k, v = m(x, a.cos(), a.sin())
    assert q.shape == (B, S, Hq, D) and k.shape == v.shape == (B, S, Hk, D)
    qkv = m.proj(x).reshape(B * S, -1)
    pq, pk = qkv[:, :Hq * D].view(-1, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(-1, Hk, D)
    want = w8.qk_norm_rope(pq, pk, qw, kw, a.cos(), a.sin(), interleaved=interleaved)
    assert same(q.reshape(-1, Hq, D), want[0]) and same(k.reshape(-1, Hk, D), want[1])
    assert same(v.reshape(-1, Hk * D), qkv[:, (Hq + Hk) * D:])
    xg = x.clone().requires_grad_()
    pos = torch.arange(B * S, dtype=torch.int32, device=DEV).reshape(B, S) % S
    out = m(xg, a.cos(), a.sin(), pos)
    assert same(out[0], q) and same(out[1], k) and same(out[2], v)
    ds = [torch.randn_like(t) for t in out]
    torch.autograd.backward(out, ds)
    gq, gk, gqw, gkw = w8.qk_norm_rope_backward(ds[0].reshape(-1, Hq, D), ds[1].reshape(-1, Hk, D), pq, pk, qw, kw,
                                                a.cos(), a.sin(), interleaved=interleaved)
    dqkv = torch.cat([gq.flatten(1), gk.flatten(1), ds[2].reshape(B * S, -1)], 1)
    dx = w8.linear_backward(dqkv, None, None, m.proj.wq, m.proj.w_scale, dw=False, dbias=False)[0]
    assert same(xg.grad.reshape(-1, K), dx)
    assert same(m.q_weight.grad, gqw.to(BF)) and same(m.k_weight.grad, gkw.to(BF))


def test_quantization_aware_training_functions(w8):
    M, N, K = 50, 40, 48
    torch.manual_seed(4)
    x, w, b = (torch.randn(*s, device=DEV).to(BF).requires_grad_() for s in ((M, K), (N, K), (N,)))
    y = w8.linear_ste(x, w, b)
    xq, xs = w8.quantize_act(x.detach())
    wq, ws = w8.quantize_weight(w.detach())
    assert same(y, w8.linear(xq, xs, wq, ws, b.detach()))
    dy = torch.randn_like(y)
    y.backward(dy)
    for t, want in zip((x, w, b), w8.linear_backward(dy, xq, xs, wq, ws)):
        assert same(t.grad, want)
    w2, b2 = (torch.randn(*s, device=DEV).to(BF).requires_grad_() for s in ((2 * N, K), (2 * N,)))
    x.grad = None
    y = w8.gated_linear_ste(x, w2, b2, "gelu")
    wq, ws = w8.quantize_weight(w2.detach())
    dy = torch.randn_like(y)
    y.backward(dy)
    for t, want in zip((x, w2, b2), w8.gated_linear_backward(dy, xq, xs, wq, ws, b2.detach(), act="gelu")):
        assert same(t.grad, want)
    # a frozen weight: only the input's gradient
    x.grad = None
    w8.linear_ste(x, w.detach(), None).sum().backward()
    assert x.grad is not None


def test_a_whole_block(w8):
    """QKV with norm and rotation, attention, output projection and gated MLP:
    one block of a transformer, against the same block in 64 bits on the
    dequantized weights and exact activations (quantization error only)."""
    B, S, C, Hq, Hk, D, F = 2, 24, 128, 4, 2, 32, 256
    proj, out, gate, up, down = linears(w8, 7, ((Hq + 2 * Hk) * D, C), (C, Hq * D), (F, C), (F, C), (C, F))
    qkv = w8.W8A8QKV(w8.W8A8Linear.from_linear(proj), Hq, Hk, torch.ones(D, device=DEV), torch.ones(D, device=DEV))
    o = w8.W8A8Linear.from_linear(out)
    mlp = w8.W8A8GatedMLP.from_linears(gate, up, down)
    a = torch.rand(S, D // 2, device=DEV) * 6

    def attend(q, k, v):
        q, k, v = (t.transpose(1, 2) for t in (q, k.repeat_interleave(Hq // Hk, 2), v.repeat_interleave(Hq // Hk, 2)))
        p = torch.softmax((q.float() @ k.float().transpose(-1, -2).contiguous()) * D ** -0.5, -1)
        return (p @ v.float().contiguous()).transpose(1, 2).reshape(B, S, Hq * D)

    def block(x):
        x = x + o(attend(*qkv(x, a.cos(), a.sin())).to(BF))
        return x + mlp(x)

    def block64(x):
        lin = lambda l, t: t @ l.weight.double().cpu().T + l.bias.double().cpu()
        r = lin(proj, x)
        parts = r.split([Hq * D, Hk * D, Hk * D], -1)
        one = torch.ones(D)
        c, s = a.cos().cpu().repeat(B, 1), a.sin().cpu().repeat(B, 1)
        q, k = (ref.norm_rope_any(t.reshape(B * S, -1, D), one, c, s, 1e-6).reshape(B, S, -1, D) for t in parts[:2])
        k, v = k.repeat_interleave(Hq // Hk, 2), parts[2].reshape(B, S, Hk, D).repeat_interleave(Hq // Hk, 2)
        q, k, v = (t.transpose(1, 2) for t in (q, k, v))
        t = (torch.softmax(q @ k.transpose(-1, -2) * D ** -0.5, -1) @ v).transpose(1, 2).reshape(B, S, Hq * D)
        x = x + lin(out, t)
        return x + lin(down, ref.act(lin(gate, x), "silu") * lin(up, x))

    x = torch.randn(B, S, C, device=DEV).to(BF).requires_grad_()
    x64 = x.detach().double().cpu().requires_grad_()
    y, y64 = block(x), block64(x64)
    dy = torch.randn_like(y)
    y.backward(dy)
    y64.backward(dy.double().cpu())
    # int8 rounding: at most half a step of amax/127 in every factor, i.e. an
    # rms of 1/sqrt(12) steps against values of about 0.3 amax: 0.8% a factor,
    # eight factors in the two sublayers' chains
    assert rel(y, y64) < 8 * 0.008 and rel(x.grad, x64.grad) < 8 * 0.008
    with torch.no_grad():
        assert same(block(x), y)


def test_backward_of_a_capture_is_refused(w8):
    lin, = linears(w8, 1, (32, 32))
    m = w8.W8A8Linear.from_linear(lin)
    x = torch.randn(4, 32, device=DEV).to(BF).requires_grad_()
    m(x).sum().backward()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    from w8a8_int8_quantized_token_amd import autograd
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        y = m(x.detach())
        with pytest.raises(RuntimeError, match="cannot be captured"):
            autograd._not_captured("this")
    g.replay()
    torch.cuda.synchronize()
    assert same(y, m(x.detach()))


# ---- graphs, streams, workspaces ----

def cases(w8, seed):
    """(name, function of a list of inputs, inputs): every entry point at a
    size of each of its paths."""
    g = torch.Generator().manual_seed(seed)

    def bf(*s):
        return torch.randn(*s, generator=g).to(BF).to(DEV)

    def q(r, k):
        return [t.to(DEV) for t in ref.codes_of(torch.randn(r, k, generator=g).to(BF))]

    out = []
    for M, N, K in [(1, 200, 512), (20, 136, 1024), (64, 256, 4096), (200, 264, 256), (33, 3000, 2048)]:
        w, s = q(N, K)
        w2, s2 = q(2 * N, K)
        b, b2 = bf(N), bf(2 * N)
        out.append((f"linear_dynamic {M}", lambda i, w=w, s=s, b=b: [w8.linear_dynamic(i[0], w, s, b)], [bf(M, K)]))
        out.append((f"gated_dynamic {M}", lambda i, w=w2, s=s2, b=b2: [w8.gated_linear_dynamic(i[0], w, s, b)],
                    [bf(M, K)]))
        xq, xs = q(M, K)
        out.append((f"linear_backward {M}", lambda i, w=w, s=s, xq=xq, xs=xs: w8.linear_backward(i[0], xq, xs, w, s),
                    [bf(M, N)]))
        out.append((f"gated_backward {M}",
                    lambda i, w=w2, s=s2, b=b2, xq=xq, xs=xs: w8.gated_linear_backward(i[0], xq, xs, w, s, b),
                    [bf(M, N)]))
    a = torch.rand(64, 32, generator=g).to(DEV) * 6
    wt = bf(64)
    out.append(("rope", lambda i: w8.qk_norm_rope(i[0], i[1], wt, wt, a.cos(), a.sin()),
                [bf(50, 8, 64), bf(50, 2, 64)]))
    out.append(("rope_backward", lambda i: w8.qk_norm_rope_backward(i[2], i[3], i[0], i[1], wt, wt, a, a),
                [bf(50, 8, 64), bf(50, 2, 64), bf(50, 8, 64), bf(50, 2, 64)]))
    return out


def equal_all(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


def test_captured_and_replayed(w8):
    for (name, f, inputs), (_, _, other) in zip(cases(w8, 1), cases(w8, 2)):
        want, want2 = f(inputs), f(other)
        static = [t.clone() for t in inputs]
        f(static)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = f(static)
        for turn in range(3):
            for src, ref_out in ((inputs, want), (other, want2)):
                for a, b in zip(static, src):
                    a.copy_(b)
                graph.replay()
                torch.cuda.synchronize()
                assert equal_all(got, ref_out), (name, turn)
                f(inputs)                       # eager work between the replays
                torch.cuda.synchronize()


def test_two_graphs_and_two_streams_at_once(w8):
    cs, ds = cases(w8, 3), cases(w8, 4)
    for (name, f, i1), (_, f2, i2) in zip(cs, ds):
        w1, w2 = f(i1), f2(i2)
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        got1, got2 = [], []
        for _ in range(4):
            with torch.cuda.stream(s1):
                got1.append(f(i1))
            with torch.cuda.stream(s2):
                got2.append(f2(i2))
        torch.cuda.synchronize()
        assert all(equal_all(g, w1) for g in got1) and all(equal_all(g, w2) for g in got2), name


def test_results_do_not_change_from_call_to_call(w8):
    for name, f, i in cases(w8, 5):
        first = f(i)
        for _ in range(5):
            assert equal_all(f(i), first), name


def test_given_workspaces(w8):
    g = torch.Generator().manual_seed(6)
    M, N, K = 100, 72, 256
    wq, ws = [t.to(DEV) for t in ref.codes_of(torch.randn(N, K, generator=g).to(BF))]
    xq, xs = [t.to(DEV) for t in ref.codes_of(torch.randn(M, K, generator=g).to(BF))]
    dy, x = torch.randn(M, N, generator=g).to(BF).to(DEV), torch.randn(M, K, generator=g).to(BF).to(DEV)
    need = w8.lib.w8a8_linear_backward_workspace(M, N, K, 1, 1, 1)
    room = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    got = w8.linear_backward(dy, xq, xs, wq, ws, workspace=room[:need])
    assert equal_all(got, w8.linear_backward(dy, xq, xs, wq, ws))
    torch.cuda.synchronize()
    assert bool((room[need:] == 0xA5).all())
    with pytest.raises(w8.W8A8Error):
        # (the size allows for a copy of dy and longer rows, which this aligned
        # dy does not need: less than its operands' own bytes)
        w8.linear_backward(dy, xq, xs, wq, ws, workspace=room[:2 * (N * K + M * N + M * K) - 16])
    need = w8.lib.w8a8_linear_dynamic_workspace(M, N, K)
    room.fill_(0xA5)
    y = w8.linear_dynamic(x, wq, ws, workspace=room[:need])
    torch.cuda.synchronize()
    assert same(y, w8.linear_dynamic(x, wq, ws)) and bool((room[need:] == 0xA5).all())


def test_outputs_end_where_they_should(w8):
    """Nothing is written before or behind the outputs, at ragged sizes."""
    g = torch.Generator().manual_seed(8)
    for M, N, K in [(1, 17, 48), (3, 33, 272), (19, 130, 64), (33, 97, 160), (130, 201, 320)]:
        wq, ws = [t.to(DEV) for t in ref.codes_of(torch.randn(2 * N, K, generator=g).to(BF))]
        x = torch.randn(M, K, generator=g).to(BF).to(DEV)
        for f, rows in ((w8.linear_dynamic, 2 * N), (w8.gated_linear_dynamic, N)):
            room = torch.full((M * rows + 64,), 7.0, dtype=BF, device=DEV)
            f(x, wq, ws, None, y=room[32:32 + M * rows].view(M, rows))
            torch.cuda.synchronize()
            assert bool((room[:32] == 7).all()) and bool((room[32 + M * rows:] == 7).all()), (M, N, K)


# ---- offsets past 32 bits ----

def test_few_tokens_over_a_weight_beyond_4_gib(w8):
    N, K, M = 66000, 65552, 2
    wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV)
    ws = torch.rand(N, device=DEV) * 1e-3
    x = torch.randn(M, K, device=DEV).to(BF)
    y = w8.linear_dynamic(x, wq, ws)
    rows = torch.cat([torch.arange(0, 40), torch.arange(N // 2, N // 2 + 40), torch.arange(N - 40, N)]).to(DEV)
    want = w8.linear(*w8.quantize_act(x), wq[rows].contiguous(), ws[rows].contiguous())
    assert same(y[:, rows], want)
    g = w8.gated_linear_dynamic(x, wq, ws)
    n = N // 2
    r = torch.cat([torch.arange(0, 40), torch.arange(n - 40, n)]).to(DEV)
    want = w8.gated_linear(*w8.quantize_act(x), wq[torch.cat([r, n + r])].contiguous(),
                           ws[torch.cat([r, n + r])].contiguous())
    assert same(g[:, r], want)


def test_gradients_beyond_4_gib(w8):
    M, N, K = 70000, 32776, 64
    wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV)
    ws = torch.rand(N, device=DEV) * 1e-2
    xq = torch.randint(-127, 128, (M, K), dtype=torch.int8, device=DEV)
    xs = torch.rand(M, device=DEV) * 1e-2
    dy = torch.randn(M, N, device=DEV, dtype=BF)
    dx, dw, db = w8.linear_backward(dy, xq, xs, wq, ws)
    rows = torch.tensor([0, 1, 35000, M - 2, M - 1], device=DEV)
    cols = torch.tensor([0, 1, 16000, N - 2, N - 1], device=DEV)
    w, x = wq.double() * ws.double()[:, None], xq.double() * xs.double()[:, None]
    assert rel(dx[rows], dy[rows].double() @ w) < 2 ** -8
    assert rel(dw[cols], dy[:, cols].double().T @ x) < 2 ** -8
    assert rel(db[cols], dy[:, cols].double().sum(0)) < 2 ** -8
    del dy, dx, dw
    # gated: the two halves of its first operands pass 4 GiB as well
    n = N // 2
    dy = torch.randn(M, n, device=DEV, dtype=BF)
    dx, dw, db = w8.gated_linear_backward(dy, xq, xs, wq, ws)
    z = xq[rows].double() @ wq.double().T * xs[rows].double()[:, None] * ws.double()
    d = torch.cat([dy[rows].double() * z[:, n:] * ref.act_slope(z[:, :n], "silu"),
                   dy[rows].double() * ref.act(z[:, :n], "silu")], 1)
    assert rel(dx[rows], d @ w) < 2 ** -8
    c = torch.tensor([0, n - 1], device=DEV)
    z = xq.double() @ wq[torch.cat([c, n + c])].double().T * xs.double()[:, None] * ws[torch.cat([c, n + c])].double()
    d = torch.cat([dy[:, c].double() * z[:, 2:] * ref.act_slope(z[:, :2], "silu"),
                   dy[:, c].double() * ref.act(z[:, :2], "silu")], 1)
    at = torch.cat([c, n + c])
    assert rel(dw[at], d.T @ x) < 2 ** -8 and rel(db[at], d.sum(0)) < 2 ** -8


def test_rope_beyond_4_gib(w8):
    M, Hq, Hk, D = 140000, 15, 2, 1024
    qkv = torch.randn(M, (Hq + Hk) * D, device=DEV, dtype=BF)
    q, k = qkv[:, :Hq * D].view(M, Hq, D), qkv[:, Hq * D:].view(M, Hk, D)
    a = torch.rand(1000, 64, device=DEV) * 6
    rows = torch.tensor([0, 1, 70000, M - 2, M - 1], device=DEV)
    keep = q[rows].clone(), k[rows].clone()
    pos = (torch.arange(M, device=DEV) % 1000).to(torch.int32)
    want = w8.qk_norm_rope(*keep, None, None, a.cos(), a.sin(), pos[rows])
    back = w8.qk_norm_rope_backward(q, k, q, k, None, None, a.cos(), a.sin(), pos, weights=False)
    want_b = w8.qk_norm_rope_backward(*keep, *keep, None, None, a.cos(), a.sin(), pos[rows], weights=False)
    assert same(back[0][rows], want_b[0]) and same(back[1][rows], want_b[1])
    w8.qk_norm_rope(q, k, None, None, a.cos(), a.sin(), q_out=q, k_out=k)
    assert same(q[rows], want[0]) and same(k[rows], want[1])


def test_native_and_checked_calls_agree(w8):
    """A plain call is one native step; with an output or workspace given the
    same call goes through the binding's checks."""
    from w8a8_int8_quantized_token_amd import _calls
    g = torch.Generator().manual_seed(9)
    M, N, K = 21, 40, 64
    wq, ws = [t.to(DEV) for t in ref.codes_of(torch.randn(2 * N, K, generator=g).to(BF))]
    xq, xs = [t.to(DEV) for t in ref.codes_of(torch.randn(M, K, generator=g).to(BF))]
    x, dy = torch.randn(M, K, generator=g).to(BF).to(DEV), torch.randn(M, N, generator=g).to(BF).to(DEV)
    b = torch.randn(2 * N, generator=g).to(BF).to(DEV)
    room = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    for act in ("silu", "gelu"):
        assert _calls.dynamic(x, wq, ws, b, {"silu": 0, "gelu": 1}[act], 2) is not None
        assert same(w8.gated_linear_dynamic(x, wq, ws, b, act=act),
                    w8.gated_linear_dynamic(x, wq, ws, b, act=act, workspace=room))
        assert equal_all(w8.gated_linear_backward(dy, xq, xs, wq, ws, b, act=act),
                         w8.gated_linear_backward(dy, xq, xs, wq, ws, b, act=act, workspace=room))
    for gelu in (False, True):
        assert same(w8.linear_dynamic(x, wq, ws, b, gelu=gelu), w8.linear_dynamic(x, wq, ws, b, gelu=gelu, workspace=room))
    dy2 = torch.cat([dy, dy], 1)
    assert _calls.backward(dy2, xq, xs, wq, ws, None, -1, True, True, True) is not None
    assert equal_all(w8.linear_backward(dy2, xq, xs, wq, ws), w8.linear_backward(dy2, xq, xs, wq, ws, workspace=room))
    q, k = torch.randn(M, 4, 32, generator=g).to(BF).to(DEV), torch.randn(M, 2, 32, generator=g).to(BF).to(DEV)
    a = torch.rand(M, 16, generator=g).to(DEV)
    w = torch.ones(32, dtype=BF, device=DEV)
    for inter in (False, True):
        args = (q, k, w, None, a.cos(), a.sin(), None, 1e-6, inter)
        assert _calls.qk_norm_rope(*args) is not None
        assert equal_all(w8.qk_norm_rope(*args), w8.qk_norm_rope(*args, q_out=torch.empty_like(q)))
        assert equal_all(w8.qk_norm_rope_backward(q, k, *args), w8.qk_norm_rope_backward(q, k, *args, workspace=room))
    # refused alike
    for bad in (lambda **o: w8.linear_dynamic(x, wq, ws[1:], None, **o), lambda **o: w8.linear_dynamic(x[:, :24], wq, ws, **o),
                lambda **o: w8.linear_backward(dy2, xq, xs[1:], wq, ws, **o)):
        for o in ({}, {"workspace": room}):
            with pytest.raises(ValueError):
                bad(**o)
    with pytest.raises(w8.W8A8Error):
        w8.linear_dynamic(x[:, :24].contiguous(), wq[:, :24].contiguous(), ws)      # K not a multiple of 16


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (17, 31, 48), (65, 40, 272), (100, 72, 256), (129, 1001, 400), (300, 2056, 512),
                                   (70, 5466, 2064), (777, 33, 144), (5, 1500, 2064), (33, 3077, 1040), (64, 750, 4112)])
def test_what_a_workspace_held_does_not_matter(w8, M, N, K):
    """Workspaces of NaNs: the padding of laid-out rows is written, not assumed."""
    g = torch.Generator().manual_seed(M + N)
    wq, ws = [t.to(DEV) for t in ref.codes_of(torch.randn(2 * N, K, generator=g).to(BF))]
    xq, xs = [t.to(DEV) for t in ref.codes_of(torch.randn(M, K, generator=g).to(BF))]
    for f, size, n, rows in ((w8.linear_backward, w8.lib.w8a8_linear_backward_workspace, 2 * N, 2 * N),
                             (w8.gated_linear_backward, w8.lib.w8a8_gated_linear_backward_workspace, N, N)):
        dy = torch.randn(M, n, generator=g).to(BF).to(DEV)
        for want in ((1, 1, 1), (1, 0, 0), (0, 1, 0)):
            flags = dict(zip(("dx", "dw", "dbias"), map(bool, want)))
            space = torch.full((size(M, rows, K, *want),), 0xFF, dtype=torch.uint8, device=DEV)
            got, fresh = f(dy, xq, xs, wq, ws, workspace=space, **flags), f(dy, xq, xs, wq, ws, **flags)
            for a, b in zip(got, fresh):
                assert (a is None) == (b is None)
                if a is not None:
                    assert bool(torch.isfinite(a).all()) and same(a, b)
