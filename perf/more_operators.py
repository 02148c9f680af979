"""Cases of the norm that leaves codes and of the adapters beside the int8
linear layer, each with a plain form in elementary torch operations:

* ``add_rms_norm_quantize``: the residual's addition, the root-mean-square norm
  of each token and its quantization (int8 or e4m3 codes with one scale per
  token), and ``add_rms_norm_backward``, its gradient with the rounding to codes
  passed straight through;
* ``linear_adapters`` and ``linear_adapters_dynamic``: the int8 linear with a
  low-rank adapter for each token, chosen by the token's index into a set of
  adapters, from codes or from bf16 activations, and
  ``linear_adapters_backward``: the gradients of the input and the adapters on
  frozen int8 weights.

``own`` chooses between the plain form and the framework's entry points.
"""
import math

import torch

own = False

# ---- cases ----------------------------------------------------------------

# ids: "runs": one request's tokens after another's, each with its own adapter;
# "own": each token's adapter drawn by itself (a decoding batch);
# "mixed": the same, and some tokens without an adapter.


def listed():
    return [
        # one decoded token between two layers: nothing but latency
        {"name": "norm_one_token", "op": "norm", "M": 1, "K": 4096, "residual": True, "fp8": False},
        # two images of 8192 tokens through a block's norm
        {"name": "norm_two_images", "op": "norm", "M": 16384, "K": 4096, "residual": True, "fp8": False},
        # a first norm (no residual yet) in front of the e4m3 linear, odd sizes
        {"name": "norm_fp8_ragged", "op": "norm", "M": 1531, "K": 5136, "residual": False, "fp8": True},
        # training: the norm's gradient with the residual stream's own
        {"name": "norm_grad", "op": "norm_grad", "M": 8192, "K": 4096, "dh": True},
        # a last norm (nothing else reads the residual stream), a ragged batch
        {"name": "norm_grad_ragged", "op": "norm_grad", "M": 777, "K": 1168, "dh": False},
        # one decoded token of a request with an adapter: latency again
        {"name": "adapters_one_token", "op": "adapters", "M": 1, "K": 2048, "N": 2048, "R": 16, "L": 4, "ids": "own",
         "bias": True, "dynamic": True},
        # a decoding batch of 16 requests, each with an adapter of its own
        {"name": "adapters_16_requests", "op": "adapters", "M": 16, "K": 4096, "N": 12288, "R": 16, "L": 64,
         "ids": "own", "bias": True, "dynamic": True},
        # prompts of 16 requests at once through a wide projection, from the codes that the norm leaves
        {"name": "adapters_prompts", "op": "adapters", "M": 8192, "K": 4096, "N": 12288, "R": 16, "L": 16,
         "ids": "runs", "bias": False, "dynamic": False},
        # sizes that fill no tile, a rank that is no power of two, tokens without an adapter between others
        {"name": "adapters_ragged", "op": "adapters", "M": 777, "K": 1168, "N": 4603, "R": 40, "L": 9, "ids": "mixed",
         "bias": True, "dynamic": False},
        # training one adapter on a frozen square projection
        {"name": "adapters_grad", "op": "adapters_grad", "M": 4096, "K": 4096, "N": 4096, "R": 16, "L": 1,
         "ids": "runs"},
        # three adapters trained at once on a batch in no order, sizes that fill no tile
        {"name": "adapters_grad_ragged", "op": "adapters_grad", "M": 1037, "K": 2064, "N": 5466, "R": 8, "L": 3,
         "ids": "mixed"},
        # four adapters of a larger rank, a full image batch
        {"name": "adapters_grad_rank_64", "op": "adapters_grad", "M": 8192, "K": 4096, "N": 8192, "R": 64, "L": 4,
         "ids": "runs"},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    """One more case of the listed ones' ranges."""
    cost = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["norm", "norm_grad", "adapters", "adapters", "adapters_grad"])
        if op == "norm":
            c = {"op": op, "M": _log_int(rng, 1, 16384), "K": _log_int(rng, 256, 12288, 16),
                 "residual": rng.random() < 0.7, "fp8": rng.random() < 0.3}
        elif op == "norm_grad":
            c = {"op": op, "M": _log_int(rng, 16, 16384), "K": _log_int(rng, 256, 12288, 16), "dh": rng.random() < 0.7}
        elif op == "adapters":
            c = {"op": op, "M": _log_int(rng, 1, 8192), "K": _log_int(rng, 256, 8192, 16), "N": _log_int(rng, 128, 12288),
                 "R": rng.choice([8, 16, 16, 32, 40, 64]), "L": _log_int(rng, 1, 64),
                 "ids": rng.choice(["runs", "runs", "own", "mixed"]), "bias": rng.random() < 0.5,
                 "dynamic": rng.random() < 0.5}
        else:
            c = {"op": op, "M": _log_int(rng, 16, 8192), "K": _log_int(rng, 256, 8192, 16), "N": _log_int(rng, 128, 12288),
                 "R": rng.choice([8, 16, 16, 32, 40, 64]), "L": _log_int(rng, 1, 8),
                 "ids": rng.choice(["runs", "runs", "own", "mixed"])}
        if _cost(c) <= cost:
            return c


def work(case):
    """Bytes (inputs once, outputs once) and operations of one pass."""
    c = case
    M, K = c["M"], c["K"]
    if c["op"] == "norm":
        per = 7 if c["residual"] else 3
        return {"bytes": per * M * K + 2 * K + 4 * M, "flops": 8 * M * K}
    if c["op"] == "norm_grad":
        return {"bytes": (8 if c["dh"] else 6) * M * K + 6 * K, "flops": 14 * M * K}
    N, R, L = c["N"], c["R"], c["L"]
    used = min(L, M)
    adapters = 2 * used * R * (K + N) + 4 * used + 4 * M
    weight = N * K + 4 * N
    low = 2 * M * R * (K + N)
    if c["op"] == "adapters":
        x = 2 * M * K if c["dynamic"] else M * K + 4 * M
        return {"bytes": x + weight + (2 * N if c["bias"] else 0) + adapters + 2 * M * N, "flops": 2 * M * N * K + low}
    # gradients: the low-rank activations and their gradients, the adapters'
    # share of the input's gradient, and the adapters' own gradients
    return {"bytes": 2 * M * N + M * K + 4 * M + weight + adapters + 2 * M * K + 2 * L * R * (K + N),
            "flops": 2 * M * N * K + 2 * low + 2 * M * R * K}


def _cost(case):
    """Work in one figure: operations, and bytes at a rate of a hundred operations each."""
    w = work(case)
    return w["flops"] + 100 * w["bytes"]


# ---- inputs ---------------------------------------------------------------


def _codes(x):
    """Rows of x to int8 codes: scale = amax / 127, code = rne(x / scale)."""
    x = x.float()
    s = x.abs().amax(1) / 127.0
    safe = torch.where(s > 0, s, torch.ones_like(s))
    q = torch.round(x / safe[:, None]).clamp(-127, 127)
    return torch.where(s[:, None] > 0, q, torch.zeros_like(q)).to(torch.int8), s


def _ids(c, g):
    M, L = c["M"], c["L"]
    if c["ids"] == "runs":
        # as many requests as adapters (or tokens), of uneven lengths
        n = min(L, M)
        ends = torch.sort(torch.rand(n, generator=g, device="cuda") * M).values
        ends[-1] = M
        run = torch.searchsorted(ends, torch.arange(M, device="cuda", dtype=torch.float32), right=True).clamp(max=n - 1)
        return torch.randperm(L, generator=g, device="cuda")[run].to(torch.int32)
    low = -1 if c["ids"] == "mixed" else 0
    return torch.randint(low, L, (M,), generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    M, K = c["M"], c["K"]
    if c["op"] in ("norm", "norm_grad"):
        h = normal(M, K)
        h[:, :: max(K // 8, 1)] *= 8.0   # a few strong channels, as a residual stream has
        st = {"case": c, "x": h.to(torch.bfloat16), "w": (1.0 + 0.2 * normal(K)).to(torch.bfloat16), "eps": 1e-6}
        if c["op"] == "norm":
            st["residual"] = (3.0 * normal(M, K)).to(torch.bfloat16) if c["residual"] else None
        else:
            st["dn"] = normal(M, K).to(torch.bfloat16)
            st["dh"] = normal(M, K).to(torch.bfloat16) if c["dh"] else None
        return st

    N, R, L = c["N"], c["R"], c["L"]
    wq, ws = _codes((normal(N, K) * 0.02).to(torch.bfloat16))
    x = normal(M, K)
    x[:, :: max(K // 8, 1)] *= 8.0
    x = x.to(torch.bfloat16)
    st = {"case": c, "wq": wq, "ws": ws, "bias": (normal(N) * 0.1).to(torch.bfloat16) if c.get("bias") else None,
          "a": (normal(L, R, K) / math.sqrt(K)).to(torch.bfloat16), "b": (normal(L, N, R) * 0.05).to(torch.bfloat16),
          "scaling": 0.5 + 1.5 * torch.rand(L, generator=g, device="cuda"), "ids": _ids(c, g)}
    if c.get("dynamic"):
        st["x"] = x
    else:
        st["xq"], st["xs"] = _codes(x)
    if c["op"] == "adapters_grad":
        st["dy"] = (normal(M, N) * 0.1).to(torch.bfloat16)
    return st


# ---- one pass -------------------------------------------------------------


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm, "norm_grad": _norm_grad, "adapters": _adapters, "adapters_grad": _adapters_grad}[
        state["case"]["op"]](state)


def _run_own(st):
    import w8a8_int8_quantized_token_amd as w8

    c = st["case"]
    if c["op"] == "norm":
        q, s, h = w8.add_rms_norm_quantize(st["x"], st["residual"], st["w"], eps=st["eps"], fp8=c["fp8"])
        if c["fp8"]:
            q = q.view(torch.float8_e4m3fn)
        return [q, s, h] if c["residual"] else [q, s]
    if c["op"] == "norm_grad":
        return list(w8.add_rms_norm_backward(st["dn"], st["x"], st["w"], eps=st["eps"], dh=st["dh"]))
    adapters = (st["a"], st["b"], st["ids"], st["scaling"])
    if c["op"] == "adapters":
        if c["dynamic"]:
            return w8.linear_adapters_dynamic(st["x"], st["wq"], st["ws"], *adapters, bias=st["bias"])
        return w8.linear_adapters(st["xq"], st["xs"], st["wq"], st["ws"], *adapters, bias=st["bias"])
    return list(w8.linear_adapters_backward(st["dy"], st["xq"], st["xs"], st["wq"], st["ws"], *adapters))


def _norm(st):
    c = st["case"]
    h = st["x"]
    if c["residual"]:
        h = (h.float() + st["residual"].float()).to(torch.bfloat16)
    hf = h.float()
    v = hf * st["w"].float()
    top = 448.0 if c["fp8"] else 127.0
    s = v.abs().amax(1) / top
    q = (v / torch.where(s > 0, s, torch.ones_like(s))[:, None]).clamp(-top, top)
    q = q.to(torch.float8_e4m3fn) if c["fp8"] else torch.round(q).to(torch.int8)
    scale = s / torch.sqrt((hf * hf).mean(1) + st["eps"])
    return [q, scale, h] if c["residual"] else [q, scale]


def _norm_grad(st):
    h, w, dn = st["x"].float(), st["w"].float(), st["dn"].float()
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + st["eps"])
    hh = h * r
    d = dn * w
    dx = r * (d - hh * (d * hh).mean(1, keepdim=True))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    return [dx.to(torch.bfloat16), (dn * hh).sum(0)]


def _x(st):
    """Codes (as fp32) and scales of the activations."""
    if "x" in st:
        q, s = _codes(st["x"])
        return q.float(), s
    return st["xq"].float(), st["xs"]


def _chosen(v, st):
    """v [M, L * R] with the columns of other adapters than the token's, and
    the tokens' scaling, applied: what is not a token's own is zero."""
    c = st["case"]
    mine = st["ids"].long()[:, None] == torch.arange(c["L"], device=v.device)
    return (v.view(-1, c["L"], c["R"]) * (mine * st["scaling"])[:, :, None]).flatten(1)


def _adapters(st):
    q, s = _x(st)
    y = (q @ st["wq"].float().t()) * s[:, None] * st["ws"]
    if st["bias"] is not None:
        y = y + st["bias"].float()
    t = _chosen((q * s[:, None]) @ st["a"].float().flatten(0, 1).t(), st)
    return (y + t @ st["b"].float().transpose(1, 2).flatten(0, 1)).to(torch.bfloat16)


def _adapters_grad(st):
    c = st["case"]
    q, s = _x(st)
    x, dy = q * s[:, None], st["dy"].float()
    a, b = st["a"].float().flatten(0, 1), st["b"].float().transpose(1, 2).flatten(0, 1)   # [L * R, K], [L * R, N]
    t, u = _chosen(x @ a.t(), st), _chosen(dy @ b.t(), st)
    dx = dy @ (st["wq"].float() * st["ws"][:, None]) + u @ a
    da = (u.t() @ x).view(c["L"], c["R"], -1)
    db = (t.t() @ dy).view(c["L"], c["R"], -1).transpose(1, 2).contiguous()
    return [v.to(torch.bfloat16) for v in (dx, da, db)]


# ---- the definitions in 64 bits -------------------------------------------


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        return _exact_norm(case, st)
    if case["op"] == "norm_grad":
        h, g, w = st["x"].to(f64), st["dn"].to(f64), st["w"].to(f64)
        n = case["K"]
        power = h.square().sum(dim=1) / n + st["eps"]
        along = torch.sum(g * w * h, dim=1)
        dx = g * w / power.sqrt().unsqueeze(1) - h * (along / (n * power ** 1.5)).unsqueeze(1)
        if case["dh"]:
            dx = dx + st["dh"].to(f64)
        return [dx, torch.sum(g * h / power.sqrt().unsqueeze(1), dim=0)]
    if case.get("dynamic"):
        # codes by definition: the fp32 scale and the fp32 quotient belong to it
        x32 = st["x"].to(torch.float32)
        scale = torch.div(x32.abs().max(dim=1, keepdim=True).values, 127.0)
        x = torch.div(x32, scale).round().to(f64) * scale.to(f64)
    else:
        x = st["xq"].to(f64) * st["xs"].to(f64).unsqueeze(1)
    w = st["wq"].to(f64) * st["ws"].to(f64).unsqueeze(1)
    a, b, scaling = st["a"].to(f64), st["b"].to(f64), st["scaling"].to(f64)
    rows = [torch.nonzero(st["ids"] == i).flatten() for i in range(case["L"])]
    if case["op"] == "adapters":
        y = torch.matmul(x, w.T)
        if st["bias"] is not None:
            y += st["bias"].to(f64)
        for i, at in enumerate(rows):
            y[at] += scaling[i] * torch.matmul(torch.matmul(x[at], a[i].T), b[i].T)
        return y
    dy = st["dy"].to(f64)
    dx, da, db = torch.matmul(dy, w), torch.zeros_like(a), torch.zeros_like(b)
    for i, at in enumerate(rows):
        u = scaling[i] * torch.matmul(dy[at], b[i])
        dx[at] += torch.matmul(u, a[i])
        da[i] = torch.matmul(u.T, x[at])
        db[i] = scaling[i] * torch.matmul(dy[at].T, torch.matmul(x[at], a[i].T))
    return [dx, da, db]


def _exact_norm(case, st):
    f64 = torch.float64
    h = st["x"]
    if case["residual"]:
        h = (h.to(f64) + st["residual"].to(f64)).to(torch.bfloat16)   # bf16 is the sum's type by definition
    v = h.to(f64) * st["w"].to(f64)
    # the codes' fp32 scale and quotient belong to their definition
    top = 448.0 if case["fp8"] else 127.0
    amax = v.abs().max(dim=1).values.to(torch.float32)
    s = torch.div(amax, top)
    q = torch.div(v.to(torch.float32), s.unsqueeze(1))
    q = q.clamp(-top, top).to(torch.float8_e4m3fn) if case["fp8"] else q.round().to(torch.int8)
    scale = amax.to(f64) / top / torch.sqrt(h.to(f64).square().mean(dim=1) + st["eps"])
    return [q, scale, h] if case["residual"] else [q, scale]
