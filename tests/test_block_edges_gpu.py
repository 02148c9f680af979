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


# ---- the QKV module ----

def qkv_module(w8, seed, norms=True):
    K, Hq, Hk, D = 64, 4, 2, 32
    torch.manual_seed(seed)
    proj = torch.nn.Linear(K, (Hq + 2 * Hk) * D, device=DEV, dtype=BF)
    w = [(1 + 0.2 * torch.randn(D, device=DEV)).to(BF) if norms else None for _ in range(2)]
    return w8.W8A8QKV(w8.W8A8Linear.from_linear(proj), Hq, Hk, *w)


def turns(P):
    a = torch.rand(P, 16, device=DEV) * 6
    return a.cos(), a.sin()


@pytest.mark.parametrize("grads", [False, True])
def test_each_sequence_of_a_batch_starts_at_position_0(w8, grads):
    """Tables longer than the sequences: a token's position is its index in
    its own sequence."""
    B, S, P = 3, 19, 64
    m = qkv_module(w8, 3)
    cos, sin = turns(P)
    x = torch.randn(2, B, S, 64, device=DEV).to(BF).requires_grad_(grads)
    with torch.set_grad_enabled(grads):
        got = m(x, cos, sin)
        for i in range(2):
            for b in range(B):
                one = m(x[i, b], cos, sin)
                for g, w in zip(got, one):
                    assert same(g[i, b], w), (i, b)
    pos = torch.arange(S, dtype=torch.int32, device=DEV).expand(2, B, S).contiguous()
    for g, w in zip(got, m(x, cos, sin, pos)):
        assert same(g, w)


def test_sequences_longer_than_the_tables(w8):
    m = qkv_module(w8, 4)
    cos, sin = turns(8)
    x = torch.randn(2, 16, 64, device=DEV).to(BF)
    with torch.no_grad():
        # whole runs of the table, in a batch or not, and one sequence alone
        flat = m(x.reshape(32, 64), cos, sin)
        for a, b in zip(m(x, cos, sin), flat):
            assert same(a.reshape(b.shape), b)
        for a, b in zip(m(x[:1, :13], cos, sin), m(x[0, :13], cos, sin)):
            assert same(a[0], b)
        # a second sequence would start inside a run
        with pytest.raises(ValueError, match="position"):
            m(x[:, :13].contiguous(), cos, sin)
        assert m(x[:, :0], cos, sin)[0].shape == (2, 0, 4, 32)
        with pytest.raises(ValueError):
            m(x, cos, sin[:7])
        with pytest.raises(TypeError):
            m(x, None, sin)
        with pytest.raises(w8.W8A8Error):
            m(x, cos[:0], sin[:0])
        # nothing to turn: no positions, whatever the tables' length
        none = torch.empty(5, 0, device=DEV)
        for a, b in zip(m(x, none, none), m(x.reshape(32, 64), none, none)):
            assert same(a.reshape(b.shape), b)


@pytest.mark.parametrize("grads", [False, True])
@pytest.mark.parametrize("norms", [False, True])
def test_what_a_hook_on_the_projection_keeps(w8, grads, norms):
    m = qkv_module(w8, 5, norms)
    cos, sin = turns(7)
    kept = []
    m.proj.register_forward_hook(lambda mod, args, out: kept.append((out, out.detach().clone())))
    x = torch.randn(2, 7, 64, device=DEV).to(BF).requires_grad_(grads)
    with torch.set_grad_enabled(grads):
        m(x, cos, sin)
    out, then = kept[0]
    assert same(out, then)


def test_gradients_that_arrive_at_odd_addresses(w8):
    m = qkv_module(w8, 6)
    cos, sin = turns(5)
    x = torch.randn(5, 64, device=DEV).to(BF).requires_grad_()
    out = m(x, cos, sin)
    ds = [torch.randn_like(t) for t in out]
    odd = [torch.empty(t.numel() + 1, dtype=BF, device=DEV)[1:].view(t.shape).copy_(t) for t in ds]
    leaves = [x, m.q_weight, m.k_weight]
    want = torch.autograd.grad(out, leaves, ds, retain_graph=True)
    got = torch.autograd.grad(out, leaves, odd)
    assert all(same(a, b) for a, b in zip(got, want))


# ---- few tokens ----

@pytest.mark.parametrize("M", [1, 3, 16, 17, 32])
@pytest.mark.parametrize("N,K", [(8448, 16), (8449, 16), (12289, 256), (2048, 256), (2049, 256), (150003, 768), (40961, 1408)])
def test_either_side_of_the_few_token_kernel(w8, M, N, K):
    """The same bits by quantize + linear, by the kernel chosen, and (up to 16
    tokens) by the few-token kernel without a workspace, or with one too small
    for the other; the largest weight has more groups of channels to a
    workgroup than their scales fit LDS at once."""
    g = torch.Generator(device=DEV).manual_seed(M + N)
    for per, f, raw in ((1, w8.linear, w8.lib.w8a8_linear_dynamic),
                        (2, w8.gated_linear, w8.lib.w8a8_gated_linear_dynamic)):
        wq = torch.randint(-127, 128, (per * N, K), generator=g, device=DEV, dtype=torch.int8)
        ws = torch.rand(per * N, generator=g, device=DEV) * 0.01
        b = torch.randn(per * N, generator=g, device=DEV).to(BF)
        x = torch.randn(M, K, generator=g, device=DEV).to(BF)
        want = f(*w8.quantize_act(x), wq, ws, b)
        assert same((w8.linear_dynamic if per == 1 else w8.gated_linear_dynamic)(x, wq, ws, b), want)
        small = torch.empty(16, dtype=torch.uint8, device=DEV)
        fits = M <= 16 and M * ((K + 127) // 128 * 128 + 16) <= 22 * 1024
        for space, size in ((None, 0), (small.data_ptr(), 16)) if fits else ():
            y = torch.full((M, N), 7.0, dtype=BF, device=DEV)
            status = raw(x.data_ptr(), wq.data_ptr(), ws.data_ptr(), b.data_ptr(), y.data_ptr(), M, N, K, 0, space,
                         size, torch.cuda.current_stream().cuda_stream)
            assert status == 0 and same(y, want)


# ---- backward nodes under a capture ----

def test_every_backward_node_refuses_a_capture(w8, monkeypatch):
    """Each node is run with the stream said to be capturing (no capture is
    made): it raises before it launches anything, and no leaf gets a gradient."""
    K = 64
    torch.manual_seed(7)
    lin = torch.nn.Linear(K, K, device=DEV, dtype=BF)
    linear = w8.W8A8Linear.from_linear(lin)
    mlp = w8.W8A8GatedMLP.from_linears(lin, lin, lin)
    qkv = qkv_module(w8, 8)
    cos, sin = turns(4)
    qkv_only = torch.randn(4, qkv.proj.out_features, device=DEV).to(BF)
    w, w2 = torch.randn(K, K, device=DEV).to(BF), torch.randn(2 * K, K, device=DEV).to(BF)

    class Projection(torch.nn.Module):      # gives the norm's node a leaf of its own
        out_features = qkv.proj.out_features

        def forward(self, x):
            return x

    alone = w8.W8A8QKV(Projection(), 4, 2, qkv.q_weight, qkv.k_weight)
    for name, f, inputs in (
            ("linear", lambda x: linear(x), [torch.randn(4, K, device=DEV).to(BF)]),
            ("mlp", lambda x: mlp(x), [torch.randn(4, K, device=DEV).to(BF)]),
            ("linear_ste", lambda x, w: w8.linear_ste(x, w), [torch.randn(4, K, device=DEV).to(BF), w]),
            ("gated_linear_ste", lambda x, w: w8.gated_linear_ste(x, w), [torch.randn(4, K, device=DEV).to(BF), w2]),
            ("qkv", lambda x: torch.cat(qkv(x, cos, sin), 1), [torch.randn(4, K, device=DEV).to(BF)]),
            ("norm", lambda x: torch.cat(alone(x, cos, sin), 1), [qkv_only])):
        leaves = [t.requires_grad_() for t in inputs]
        y = f(*leaves).sum()
        with monkeypatch.context() as p:
            p.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
            with pytest.raises(RuntimeError, match="cannot be captured"):
                y.backward()
        torch.cuda.synchronize()
        assert all(t.grad is None for t in leaves), name
        f(*leaves).sum().backward()
        assert all(t.grad is not None for t in leaves), name
    assert qkv.q_weight.grad is not None and alone.q_weight.grad is not None
