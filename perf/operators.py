"""Cases of the operators around the int8 linear layer, each with a plain form
in elementary torch operations:

* ``linear_dynamic``: bf16 activations of a few tokens in, the quantization of
  each token, the int8 product, scales, bias (and GELU), bf16 out;
* ``gated_linear_dynamic``: the same for the gate and up projections of a gated
  feed-forward block with act(gate) * up;
* ``linear_backward`` and ``gated_linear_backward``: the gradients of both with
  the rounding to codes passed straight through, for the input alone (frozen
  weights) or for the input, the weight and the bias;
* ``qk_norm_rope`` and ``qk_norm_rope_backward``: RMS norms of each head's
  query and key with the position rotation, and their gradient.

``own`` chooses between the plain form and the framework's entry points.
"""
import math

import torch

own = False

# ---- cases ----------------------------------------------------------------


def listed():
    return [
        # sampling with one conditioning token through a small projection:
        # nothing but latency
        {"name": "linear_one_token", "op": "linear", "M": 1, "K": 2048, "N": 2048, "bias": True, "gelu": False},
        # a handful of tokens (a small serving batch) through a wide
        # up-projection with GELU: the weights' bytes are the floor
        {"name": "linear_16_tokens_gelu", "op": "linear", "M": 16, "K": 4096, "N": 12288, "bias": True, "gelu": True},
        # one token through the gated block's first half
        {"name": "gated_one_token", "op": "gated", "M": 1, "K": 4096, "N": 12288, "bias": False, "act": "silu"},
        # a full image batch (8192 tokens) through the gated block's first half
        {"name": "gated_8192_tokens", "op": "gated", "M": 8192, "K": 4096, "N": 12288, "bias": True, "act": "silu"},
        # training with straight-through rounding: all gradients of a square
        # projection
        {"name": "linear_grad", "op": "linear_grad", "M": 4096, "K": 4096, "N": 4096, "dw": True},
        # adapters on frozen int8 weights: a ragged batch, input gradient only
        {"name": "linear_grad_frozen_ragged", "op": "linear_grad", "M": 777, "K": 1168, "N": 4603, "dw": False},
        # all gradients of a gated block's first half
        {"name": "gated_grad", "op": "gated_grad", "M": 4096, "K": 2048, "N": 8192, "bias": True, "act": "silu", "dw": True},
        # its input gradient on frozen weights, sizes that fill no tile
        {"name": "gated_grad_frozen_ragged", "op": "gated_grad", "M": 1037, "K": 2064, "N": 5466, "bias": False, "act": "gelu", "dw": False},
        # one token's queries and keys out of a packed QKV row
        {"name": "rope_one_token", "op": "rope", "M": 1, "P": 4096, "Hq": 32, "Hk": 8, "D": 128, "rot": 128, "interleaved": False, "positions": True},
        # a full image batch's queries and keys (two images of 8192 tokens)
        {"name": "rope_two_images", "op": "rope", "M": 16384, "P": 8192, "Hq": 24, "Hk": 24, "D": 128, "rot": 128, "interleaved": True, "positions": False},
        # the gradient of the same, smaller, with shared key heads
        {"name": "rope_grad", "op": "rope_grad", "M": 8192, "P": 4096, "Hq": 32, "Hk": 8, "D": 128, "rot": 128, "interleaved": False, "positions": False},
        # ragged rows, a head size that is no power of two, a partial rotation
        {"name": "rope_grad_partial_ragged", "op": "rope_grad", "M": 1531, "P": 2000, "Hq": 10, "Hk": 2, "D": 80, "rot": 32, "interleaved": True, "positions": True},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    """One more case of the listed ones' ranges."""
    cost = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["linear", "gated", "linear_grad", "gated_grad", "rope", "rope_grad"])
        if op == "linear":
            c = {"op": op, "M": _log_int(rng, 1, 32), "K": _log_int(rng, 256, 12288, 16), "N": _log_int(rng, 128, 16384),
                 "bias": rng.random() < 0.5, "gelu": rng.random() < 0.5}
        elif op == "gated":
            c = {"op": op, "M": _log_int(rng, 1, 8192), "K": _log_int(rng, 256, 8192, 16), "N": _log_int(rng, 128, 16384),
                 "bias": rng.random() < 0.5, "act": rng.choice(["silu", "gelu"])}
        elif op == "linear_grad":
            c = {"op": op, "M": _log_int(rng, 16, 8192), "K": _log_int(rng, 256, 8192, 16), "N": _log_int(rng, 128, 12288),
                 "dw": rng.random() < 0.5}
        elif op == "gated_grad":
            c = {"op": op, "M": _log_int(rng, 16, 8192), "K": _log_int(rng, 256, 8192, 16), "N": _log_int(rng, 128, 12288),
                 "bias": rng.random() < 0.5, "act": rng.choice(["silu", "gelu"]), "dw": rng.random() < 0.5}
        else:
            D = rng.choice([32, 64, 80, 96, 128, 192, 256])
            Hk = rng.choice([1, 2, 3, 4, 8, 16])
            c = {"op": op, "M": _log_int(rng, 1, 16384), "P": rng.randint(100, 9000), "Hq": Hk * rng.choice([1, 2, 3, 4, 5]),
                 "Hk": Hk, "D": D, "rot": rng.choice([D, D, D // 2 // 16 * 16 or 16]), "interleaved": rng.random() < 0.5,
                 "positions": rng.random() < 0.5}
        if _cost(c) <= cost:
            return c


def work(case):
    """Bytes (inputs once, outputs once) and operations of one pass."""
    c = case
    if c["op"].startswith("rope"):
        back = c["op"] == "rope_grad"
        heads = c["Hq"] + c["Hk"]
        values = c["M"] * heads * c["D"]
        table = min(c["M"], c["P"]) * c["rot"] * 4 + (c["M"] * 4 if c["positions"] else 0)
        return {"bytes": values * (6 if back else 4) + table + c["D"] * (12 if back else 4),
                "flops": values * (16 if back else 8)}
    M, K = c["M"], c["K"]
    cols = c["N"] * (2 if c["op"].startswith("gated") else 1)   # rows of the weight
    weight = cols * K + 4 * cols
    product = 2 * M * K * cols
    bias = 2 * cols if c.get("bias") else 0
    if c["op"] in ("linear", "gated"):
        return {"bytes": 2 * M * K + weight + bias + 2 * M * c["N"], "flops": product}
    # gradients: dy and the weight are read and dx written; for a gated block
    # the product is needed again (from the activation codes); the weight's
    # gradient needs the codes and is written with the bias's
    gated, dw = c["op"] == "gated_grad", c["dw"]
    codes = M * K + 4 * M if gated or dw else 0
    return {"bytes": 2 * M * c["N"] + weight + bias + codes + 2 * M * K + ((2 * cols * K + 2 * cols) if dw else 0),
            "flops": product * (1 + int(gated) + int(dw))}


def _cost(case):
    """Work in one figure: operations, and bytes at a rate of a hundred operations each."""
    w = work(case)
    return w["flops"] + 100 * w["bytes"]


# ---- inputs ---------------------------------------------------------------


def _quantize(x):
    """Rows of x to int8 codes: scale = amax / 127, code = rne(x / scale)."""
    x = x.float()
    s = x.abs().amax(1) / 127.0
    safe = torch.where(s > 0, s, torch.ones_like(s))
    q = torch.round(x / safe[:, None]).clamp(-127, 127)
    return torch.where(s[:, None] > 0, q, torch.zeros_like(q)), s


def _codes(x):
    q, s = _quantize(x)
    return q.to(torch.int8), s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if c["op"].startswith("rope"):
        M, Hq, Hk, D = c["M"], c["Hq"], c["Hk"], c["D"]
        # queries, keys and values side by side, as a QKV projection leaves them
        qkv = (normal(M, (Hq + 2 * Hk) * D) * 2.0).to(torch.bfloat16)
        half = c["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        angle = torch.arange(c["P"], dtype=torch.float64, device="cuda")[:, None] * freq
        st = {"case": c, "q": qkv[:, :Hq * D].view(M, Hq, D), "k": qkv[:, Hq * D:(Hq + Hk) * D].view(M, Hk, D),
              "qw": (1.0 + 0.2 * normal(D)).to(torch.bfloat16), "kw": (1.0 + 0.2 * normal(D)).to(torch.bfloat16),
              "cos": angle.cos().float().contiguous(), "sin": angle.sin().float().contiguous(), "eps": 1e-6,
              "positions": torch.randint(0, c["P"], (M,), generator=g, device="cuda", dtype=torch.int32)
              if c["positions"] else None}
        if c["op"] == "rope_grad":
            st["dq"] = normal(M, Hq, D).to(torch.bfloat16)
            st["dk"] = normal(M, Hk, D).to(torch.bfloat16)
        return st

    M, K, N = c["M"], c["K"], c["N"]
    rows = N * (2 if c["op"].startswith("gated") else 1)
    wq, ws = _codes((normal(rows, K) * 0.02).to(torch.bfloat16))
    st = {"case": c, "wq": wq, "ws": ws,
          "bias": (normal(rows) * 0.1).to(torch.bfloat16) if c.get("bias") else None}
    x = normal(M, K)
    x[:, :: max(K // 8, 1)] *= 8.0   # a few strong channels, as activations have
    x = x.to(torch.bfloat16)
    if c["op"].endswith("grad"):
        # what the forward pass keeps: the codes and their scales
        st["xq"], st["xs"] = _codes(x)
        st["dy"] = (normal(M, N) * 0.1).to(torch.bfloat16)
    else:
        st["x"] = x
    return st


# ---- one pass -------------------------------------------------------------


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    return {"linear": _linear, "gated": _gated, "linear_grad": _linear_grad, "gated_grad": _gated_grad,
            "rope": _rope, "rope_grad": _rope_grad}[c["op"]](state)


def _run_own(st):
    import w8a8_int8_quantized_token_amd as w8

    c = st["case"]
    if c["op"] == "linear":
        return w8.linear_dynamic(st["x"], st["wq"], st["ws"], st["bias"], gelu=c["gelu"])
    if c["op"] == "gated":
        return w8.gated_linear_dynamic(st["x"], st["wq"], st["ws"], st["bias"], act=c["act"])
    if c["op"] == "linear_grad":
        r = w8.linear_backward(st["dy"], st["xq"], st["xs"], st["wq"], st["ws"], dw=c["dw"], dbias=c["dw"])
        return [t for t in r if t is not None]
    if c["op"] == "gated_grad":
        r = w8.gated_linear_backward(st["dy"], st["xq"], st["xs"], st["wq"], st["ws"], st["bias"], act=c["act"],
                                     dw=c["dw"], dbias=c["dw"])
        return [t for t in r if t is not None]
    if c["op"] == "rope":
        return w8.qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], st["cos"], st["sin"], st["positions"],
                               eps=st["eps"], interleaved=c["interleaved"])
    return w8.qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], st["qw"], st["kw"], st["cos"], st["sin"],
                                    st["positions"], eps=st["eps"], interleaved=c["interleaved"])


def _phi(v):
    return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5)))


def _act(v, act):
    return v / (1.0 + torch.exp(-v)) if act == "silu" else v * _phi(v)


def _act_grad(v, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-v))
        return s * (1.0 + v * (1.0 - s))
    return _phi(v) + v * torch.exp(-0.5 * v * v) * (1.0 / math.sqrt(2.0 * math.pi))


def _scaled(q, s, wq, ws, bias):
    """The int8 product in 32 bits with its scales and bias."""
    y = (q @ wq.float().t()) * s[:, None] * ws
    return y if bias is None else y + bias.float()


def _linear(st):
    q, s = _quantize(st["x"])
    y = _scaled(q, s, st["wq"], st["ws"], st["bias"])
    return (y * _phi(y) if st["case"]["gelu"] else y).to(torch.bfloat16)


def _gated(st):
    q, s = _quantize(st["x"])
    g, u = _scaled(q, s, st["wq"], st["ws"], st["bias"]).chunk(2, dim=1)
    return (_act(g, st["case"]["act"]) * u).to(torch.bfloat16)


def _product_grads(d, st):
    """Gradients of the scaled product for d [M, rows]: input, weight, bias."""
    dx = (d @ (st["wq"].float() * st["ws"][:, None])).to(torch.bfloat16)
    if not st["case"]["dw"]:
        return [dx]
    dw = d.t() @ (st["xq"].float() * st["xs"][:, None])
    return [dx, dw.to(torch.bfloat16), d.sum(0).to(torch.bfloat16)]


def _linear_grad(st):
    return _product_grads(st["dy"].float(), st)


def _gated_grad(st):
    act, dy = st["case"]["act"], st["dy"].float()
    g, u = _scaled(st["xq"].float(), st["xs"], st["wq"], st["ws"], st["bias"]).chunk(2, dim=1)
    return _product_grads(torch.cat([dy * u * _act_grad(g, act), dy * _act(g, act)], dim=1), st)


def _tables(st):
    """cos and sin of each row, [M, 1, rot / 2]."""
    rows = torch.arange(st["q"].shape[0], device="cuda") % st["cos"].shape[0]
    if st["positions"] is not None:
        rows = st["positions"].long()
    return st["cos"][rows][:, None], st["sin"][rows][:, None]


def _rotate(x, cos, sin, interleaved):
    """The first 2 * cos.shape[-1] values of each head rotated pairwise."""
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], dim=-1).flatten(-2) if interleaved else torch.cat([ra, rb], dim=-1)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1)


def _rope(st):
    cos, sin = _tables(st)

    def one(x, w):
        x = x.float()
        n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w.float()
        return _rotate(n, cos, sin, st["case"]["interleaved"]).to(torch.bfloat16)

    return [one(st["q"], st["qw"]), one(st["k"], st["kw"])]


def _rope_grad(st):
    cos, sin = _tables(st)

    def one(dy, x, w):
        x, w = x.float(), w.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"])
        xh = x * r
        dn = _rotate(dy.float(), cos, -sin, st["case"]["interleaved"])   # the rotation back
        dh = dn * w
        dx = r * (dh - xh * (dh * xh).mean(-1, keepdim=True))
        return dx.to(torch.bfloat16), (dn * xh).sum((0, 1))

    dq, dqw = one(st["dq"], st["q"], st["qw"])
    dk, dkw = one(st["dk"], st["k"], st["kw"])
    return [dq, dk, dqw, dkw]


# ---- the definitions in 64 bits -------------------------------------------


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"].startswith("rope"):
        return _exact_rope(case, st)
    wd = st["wq"].to(f64) * st["ws"].to(f64).unsqueeze(1)
    b = 0.0 if st["bias"] is None else st["bias"].to(f64)
    if case["op"].endswith("grad"):
        xd = st["xq"].to(f64) * st["xs"].to(f64).unsqueeze(1)
    else:
        # codes by definition: the fp32 scale and the fp32 quotient belong to it
        x = st["x"].to(torch.float32)
        scale = torch.div(x.abs().max(dim=1, keepdim=True).values, 127.0)
        quotient = torch.div(x, scale)   # no row of the inputs is all zeros
        xd = quotient.round().to(f64) * scale.to(f64)

    def gauss(v):
        return torch.special.ndtr(v)

    def act(v):
        return v * torch.sigmoid(v) if case["act"] == "silu" else v * gauss(v)

    if case["op"] == "linear":
        z = torch.matmul(xd, wd.T) + b
        return z * gauss(z) if case["gelu"] else z
    if case["op"] == "gated":
        z = torch.matmul(xd, wd.T) + b
        n = case["N"]
        return act(z[:, :n]) * z[:, n:]
    d = st["dy"].to(f64)
    if case["op"] == "gated_grad":
        z = torch.matmul(xd, wd.T) + b
        n = case["N"]
        gate, up = z[:, :n], z[:, n:]
        if case["act"] == "silu":
            s = torch.sigmoid(gate)
            slope = s + gate * s * torch.sigmoid(-gate)
        else:
            slope = gauss(gate) + gate * torch.exp(-gate.square() / 2) / math.sqrt(2 * math.pi)
        d = torch.cat((d * up * slope, d * act(gate)), 1)
    out = [torch.matmul(d, wd)]
    if case["dw"]:
        out += [torch.matmul(d.T, xd), d.sum(dim=0)]
    return out


def _exact_rope(case, st):
    f64 = torch.float64
    M, rot, D = case["M"], case["rot"], case["D"]
    where = torch.remainder(torch.arange(M, device="cuda"), case["P"]) if st["positions"] is None else st["positions"].long()
    # each rotation as a complex factor; values past the rotation stay
    turn = torch.complex(st["cos"].to(f64)[where], st["sin"].to(f64)[where]).unsqueeze(1)

    def pairs(v):
        v = v[..., :rot].reshape(*v.shape[:-1], rot // 2, 2) if case["interleaved"] else \
            v[..., :rot].reshape(*v.shape[:-1], 2, rot // 2).transpose(-1, -2)
        return torch.view_as_complex(v.contiguous())

    def turned(v, factor):
        p = torch.view_as_real(pairs(v) * factor)
        p = p if case["interleaved"] else p.transpose(-1, -2)
        return torch.cat((p.reshape(*v.shape[:-1], rot), v[..., rot:]), dim=-1)

    def inverse_rms(x):
        return 1.0 / torch.sqrt(x.square().sum(-1, keepdim=True) / D + st["eps"])

    if case["op"] == "rope":
        return [turned(x.to(f64) * inverse_rms(x.to(f64)) * w.to(f64), turn)
                for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"]))]
    dxs, dws = [], []
    for dy, x, w in ((st["dq"], st["q"], st["qw"]), (st["dk"], st["k"], st["kw"])):
        x, w = x.to(f64), w.to(f64)
        r = inverse_rms(x)
        dn = turned(dy.to(f64), turn.conj())
        along = (dn * w * x).sum(-1, keepdim=True)
        dxs.append(dn * w * r - x * along * r ** 3 / D)
        dws.append((dn * x * r).sum(dim=(0, 1)))
    return dxs + dws
