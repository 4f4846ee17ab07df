"""Measured cases of the operators between a layer's projections and its attention:
the norm of Q and K over each head with the position rotation in the same pass, and
the linear layer with bias, activation and residual in its epilogue; each forward
and backward.

``run`` computes a case in elementary torch operations (fp32, one rounding at the
end) where ``own`` is false, and calls the library where it is true.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------ the cases
def _norm(name, grad, B, Hq, Hk, F, h, w, text, d, axes, halves, dtype, wdtype):
    c = {"op": "norm_rope", "grad": grad, "B": B, "Hq": Hq, "Hk": Hk, "F": F, "h": h, "w": w, "text": text, "d": d,
         "at": axes[0], "ah": axes[1], "aw": axes[2], "halves": halves, "dtype": dtype, "wdtype": wdtype}
    return {"name": name, **c} if name else c


def _linear(name, grad, B, N, in_heads, in_dim, out_heads, out_dim, act, bias, residual, pre, dtype):
    c = {"op": "linear", "grad": grad, "B": B, "N": N, "in_heads": in_heads, "in_dim": in_dim, "out_heads": out_heads,
         "out_dim": out_dim, "act": act, "bias": bias, "residual": residual, "pre": pre, "dtype": dtype}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one new token of a few requests, each at its own far position: latency counts
        _norm("norm_rope_token", False, 4, 16, 4, 1, 1, 1, 1, 128, (128, 0, 0), True, "bf16", "bf16"),
        # Q and K of one 480p layer (21 frames of 30 x 52 latents), slices of the fused projection in,
        # the attention's head-major layout out
        _norm("norm_rope_480p", False, 1, 24, 24, 21, 30, 52, 0, 128, (44, 42, 42), False, "bf16", "fp32"),
        # text before the latents, fewer key heads than query heads, an odd token count, fp16
        _norm("norm_rope_text_fp16", False, 2, 10, 2, 3, 33, 41, 37, 64, (16, 24, 24), True, "fp16", "fp16"),
        # a 720p layer's training step: gradients of the projections and of both norms' weights
        _norm("norm_rope_grad_720p", True, 1, 24, 24, 21, 45, 80, 0, 128, (32, 48, 48), True, "bf16", "fp32"),
        # the same for a small fp32 layer whose axes leave channels unrotated
        _norm("norm_rope_grad_fp32", True, 2, 5, 5, 3, 23, 31, 9, 96, (16, 24, 24), False, "fp32", "fp32"),
        # the embedding of a denoising step: two rows through one small layer, latency counts
        _linear("linear_embed", False, 2, 1, 0, 256, 0, 2048, "silu", True, False, False, "bf16"),
        # two prompts of odd length into the model's width
        _linear("linear_text", False, 2, 333, 0, 4096, 0, 2048, "gelu_tanh", True, False, False, "bf16"),
        # Q, K and V of a 480p layer of 16 heads, written head-major as the attention reads them
        _linear("linear_qkv_480p", False, 1, 32760, 0, 2048, 48, 128, "", True, False, False, "bf16"),
        # the attention's head-major output through its projection, onto the residual stream
        _linear("linear_out_480p", False, 1, 32760, 16, 128, 0, 2048, "", True, True, False, "bf16"),
        # the wide half of the layer's feed-forward in training: the pre-activations are kept
        _linear("linear_wide_480p", False, 1, 32760, 0, 2048, 0, 8192, "gelu_tanh", True, False, True, "bf16"),
        # gradients of a small layer of odd sizes, fp16
        _linear("linear_grad_odd", True, 3, 1667, 0, 1160, 0, 1544, "silu", True, False, True, "fp16"),
        # gradients of the wide feed-forward layer
        _linear("linear_grad_480p", True, 1, 32760, 0, 2048, 0, 8192, "gelu_tanh", True, False, True, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if rng.random() < 0.45:
        d = rng.choice([64, 64, 128, 128, 80, 96, 256])
        half = d // 2
        ah = 2 * rng.randint(1, half // 2)
        aw = 2 * rng.randint(1, half // 2 - 1)
        room = d - ah - aw
        at = rng.choice([room, 2 * rng.randint(1, room // 2)])
        H = rng.randint(1, 16)
        return _norm("", rng.random() < 0.5, rng.choice([1, 1, 2, 3]), H, rng.choice([H, max(1, H // 4)]),
                     _log_int(rng, 1, 21), _log_int(rng, 1, 45), _log_int(rng, 1, 80), rng.choice([0, 0, rng.randint(1, 300)]),
                     d, (at, ah, aw), rng.random() < 0.5, dtype, rng.choice([dtype, "fp32"]))
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    B, N = rng.choice([1, 1, 2, 3]), _log_int(rng, 1, 32760)
    in_heads, out_heads = rng.choice([0, 0, 0, rng.randint(1, 24)]), rng.choice([0, 0, rng.randint(1, 48)])
    in_dim = rng.choice([64, 128]) if in_heads else 8 * _log_int(rng, 8, 640)
    out_dim = rng.choice([64, 128]) if out_heads else 8 * _log_int(rng, 8, 1024)
    # no more products than the largest listed case
    most = 32760 * 2048 * 8192 // (max(1, in_heads) * in_dim * max(1, out_heads) * out_dim)
    N = max(1, min(N, most // B))
    act = rng.choice(["", "gelu", "gelu_tanh", "silu"])
    if rng.random() < 0.45:
        return _linear("", True, B, N, in_heads, in_dim, out_heads, out_dim, act, rng.random() < 0.7, False, bool(act), dtype)
    return _linear("", False, B, N, in_heads, in_dim, out_heads, out_dim, act, rng.random() < 0.7, rng.random() < 0.4,
                   bool(act) and rng.random() < 0.5, dtype)


# ------------------------------------------------------------------ the inputs
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


def _axes(c):
    return [a for a in (c["at"], c["ah"], c["aw"]) if a]


def _tokens(c):
    # the case of single tokens has its text token alone
    return c["text"] if _single(c) else c["text"] + c["F"] * c["h"] * c["w"]


def _single(c):
    return c["text"] == c["F"] * c["h"] * c["w"] == 1


def _positions(c, g):
    """None (the latents' grid), or int32 [N, axes] / [B, N, axes]."""
    if not c["text"]:
        return None
    axes, B = len(_axes(c)), c["B"]
    if _single(c):
        return torch.randint(0, 100000, (B, 1, 1), generator=g, device="cuda").expand(B, 1, axes).to(torch.int32).contiguous()
    t = torch.arange(c["F"] * c["h"] * c["w"], device="cuda")
    video = torch.stack([t // (c["h"] * c["w"]) + c["text"], t // c["w"] % c["h"], t % c["w"]], 1)
    start = torch.randint(0, 100000, (1,), generator=g, device="cuda")
    text = (torch.arange(c["text"], device="cuda") + start)[:, None].expand(-1, 3)
    return torch.cat([text, video]).to(torch.int32).contiguous()


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, dt = case, DTYPES[case["dtype"]]
    s = {"case": case}
    if c["op"] == "norm_rope":
        B, d, n, Hq, Hk = c["B"], c["d"], _tokens(c), c["Hq"], c["Hk"]
        s["positions"], s["grid"] = _positions(c, g), (c["F"], c["h"], c["w"])
        # the heads of a fused projection [B, N, Hq + 2 Hk, d], of different sizes
        size = torch.exp(0.5 * _randn(g, Hq + 2 * Hk, 1))
        proj = (_randn(g, B, n, Hq + 2 * Hk, d) * size).to(dt)
        s["x"] = [proj[:, :, :Hq].transpose(1, 2), proj[:, :, Hq:Hq + Hk].transpose(1, 2)]
        s["weight"] = [(1 + 0.2 * _randn(g, d)).to(DTYPES[c["wdtype"]]) for _ in range(2)]
        if c["grad"]:
            s["dout"] = [_randn(g, B, H, n, d).to(dt) for H in (Hq, Hk)]
        return s
    B, N = c["B"], c["N"]
    K, M = max(1, c["in_heads"]) * c["in_dim"], max(1, c["out_heads"]) * c["out_dim"]
    like = lambda heads, dim: _randn(g, *((B, heads, N, dim) if heads else (B, N, dim))).to(dt)
    s["x"] = like(c["in_heads"], c["in_dim"])
    s["weight"] = (_randn(g, M, K) / math.sqrt(K)).to(dt)
    s["bias"] = (0.5 * _randn(g, M)).to(dt) if c["bias"] else None
    s["residual"] = like(c["out_heads"], c["out_dim"]) if c["residual"] else None
    if c["grad"]:
        s["dout"] = like(c["out_heads"], c["out_dim"])
        s["pre"] = like(c["out_heads"], c["out_dim"]) if c["act"] else None
    return s


# --------------------------------------------------------- the library's calls
def _norm_own(s):
    import block_sparse_attention_tsr_gb300 as tsr
    c = s["case"]
    kw = dict(axis_dims=_axes(c), eps=EPS, theta=THETA, halves=c["halves"])
    if s["positions"] is not None:
        kw["positions"] = s["positions"]
    else:
        kw["grid"] = s["grid"]
    if not c["grad"]:
        return tsr.tsr_norm_rope(s["x"], s["weight"], **kw)
    # gradients go back to the projections' token-major layout
    out = [torch.empty((c["B"], x.shape[2], x.shape[1], c["d"]), dtype=x.dtype, device=x.device) for x in s["x"]]
    _, dweight = tsr.tsr_norm_rope_backward(s["dout"], s["x"], s["weight"], out=[o.transpose(1, 2) for o in out], **kw)
    return out + dweight


def _linear_own(s):
    import block_sparse_attention_tsr_gb300 as tsr
    c = s["case"]
    act = c["act"] or None
    if c["grad"]:
        dx, dw, db = tsr.tsr_linear_backward(s["dout"], s["x"], s["weight"], activation=act, pre=s["pre"],
                                             need=(True, True, c["bias"]))
        return [dx, dw] + ([db] if c["bias"] else [])
    return tsr.tsr_linear(s["x"], s["weight"], s["bias"], activation=act, residual=s["residual"],
                          heads=c["out_heads"], pre=True if c["pre"] else None)


# -------------------------------------------------------------- the plain forms
def _angles(s):
    """cos and sin [N, pairs] (or [B, 1, N, pairs]): position x frequency in 64 bits, so
    that far positions keep their place on the circle."""
    c, pos = s["case"], s["positions"]
    if pos is None:
        F, h, w = s["grid"]
        t = torch.arange(F * h * w, device="cuda")
        pos = torch.stack([t // (h * w), t // w % h, t % w], 1)
    parts = []
    for axis, width in enumerate(_axes(c)):
        j = torch.arange(width // 2, device="cuda", dtype=torch.float64)
        parts.append(pos[..., axis, None].double() * THETA ** (-2 * j / width))
    a = torch.cat(parts, -1)
    if a.dim() == 3:
        a = a[:, None]
    return torch.cos(a).float(), torch.sin(a).float()


def _pair_places(s):
    """The channels of each pair's first and second element."""
    first, second, at = [], [], 0
    for width in _axes(s["case"]):
        j = torch.arange(width // 2, device="cuda")
        first.append(at + (j if s["case"]["halves"] else 2 * j))
        second.append(at + (j + width // 2 if s["case"]["halves"] else 2 * j + 1))
        at += width
    return torch.cat(first), torch.cat(second)


def _turn(y, cos, sin, i, j):
    """A copy of y whose pairs (i, j) are turned."""
    z = y.clone()
    a, b = y[..., i], y[..., j]
    z[..., i] = a * cos - b * sin
    z[..., j] = a * sin + b * cos
    return z


def _norm_plain(s):
    c = s["case"]
    (cos, sin), (i, j) = _angles(s), _pair_places(s)
    if not c["grad"]:
        out = []
        for x, w in zip(s["x"], s["weight"]):
            y = x.float()
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
            out.append(_turn(y, cos, sin, i, j).to(x.dtype).contiguous())
        return out
    dxs, dws = [], []
    for x, w, dout in zip(s["x"], s["weight"], s["dout"]):
        x32 = x.float()
        r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
        xhat = x32 * r
        g = _turn(dout.float(), cos, -sin, i, j)
        dws.append((g * xhat).sum((0, 1, 2)).to(w.dtype))
        g = g * w.float()
        dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        dxs.append(dx.to(x.dtype).transpose(1, 2).contiguous())
    return dxs + dws


def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def _rows(t):
    """[B, N, features] of a token-major or head-major tensor."""
    return t.transpose(1, 2).flatten(2) if t.dim() == 4 else t


def _back(y, heads, like):
    """The layout a result is returned in."""
    y = y.to(like.dtype)
    return y.unflatten(2, (heads, -1)).transpose(1, 2).contiguous() if heads else y


def _linear_plain(s):
    c = s["case"]
    x, w = _rows(s["x"]).float(), s["weight"].float()
    if not c["grad"]:
        z = x @ w.t()
        if c["bias"]:
            z = z + s["bias"].float()
        y = _act(z, c["act"])
        if c["residual"]:
            y = y + _rows(s["residual"]).float()
        out = _back(y, c["out_heads"], s["x"])
        return (out, _back(z, c["out_heads"], s["x"])) if c["pre"] else out
    dz = _rows(s["dout"]).float()
    if c["act"]:
        dz = dz * _act_slope(_rows(s["pre"]).float(), c["act"])
    flat = dz.flatten(0, 1)
    grads = [_back(dz @ w, c["in_heads"], s["x"]), (flat.t() @ x.flatten(0, 1)).to(s["weight"].dtype)]
    return grads + ([flat.sum(0).to(s["weight"].dtype)] if c["bias"] else [])


def run(state):
    if state["case"]["op"] == "norm_rope":
        return _norm_own(state) if own else _norm_plain(state)
    return _linear_own(state) if own else _linear_plain(state)


# --------------------------------------------------------------- the work
def work(case):
    c = case
    es = SIZES[c["dtype"]]
    if c["op"] == "norm_rope":
        n = _tokens(c)
        values = c["B"] * (c["Hq"] + c["Hk"]) * n * c["d"]
        positions = 4 * len(_axes(c)) * n if c["text"] else 0
        weights = 2 * c["d"] * SIZES[c["wdtype"]]
        if c["grad"]:
            return {"bytes": 3 * values * es + positions + 2 * weights, "flops": 14 * values}
        return {"bytes": 2 * values * es + positions + weights, "flops": 7 * values}
    T = c["B"] * c["N"]
    K, M = max(1, c["in_heads"]) * c["in_dim"], max(1, c["out_heads"]) * c["out_dim"]
    if c["grad"]:
        # dout, pre, x and the weight in; dx, dweight and dbias out
        moved = T * M * (1 + bool(c["act"])) + 2 * T * K + 2 * M * K + M * c["bias"]
        return {"bytes": moved * es, "flops": 4 * T * K * M}
    moved = T * K + M * K + T * M * (1 + c["residual"] + c["pre"]) + M * c["bias"]
    return {"bytes": moved * es, "flops": 2 * T * K * M}


# ------------------------------------------------------- the definition, 64 bits
def _exact_turn(s, x, back):
    """x [B, H, N, d] (64 bits) turned in the complex plane."""
    c = s["case"]
    if s["positions"] is None:
        pos = torch.cartesian_prod(*(torch.arange(n, device="cuda", dtype=torch.float64) for n in s["grid"])).view(-1, 3)
    else:
        pos = s["positions"].double()
    pieces, at = [], 0
    for axis, width in enumerate(_axes(c)):
        part = x[..., at:at + width]
        at += width
        pair = part.unflatten(-1, (2, width // 2)).transpose(-1, -2) if c["halves"] else part.unflatten(-1, (-1, 2))
        speed = torch.exp(torch.arange(0, width, 2, device="cuda", dtype=torch.float64) * (-math.log(THETA) / width))
        angle = pos[..., axis, None] * speed
        angle = angle[:, None] if angle.dim() == 3 else angle
        turn = torch.polar(torch.ones_like(angle), -angle if back else angle)
        pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        pieces.append((pair.transpose(-1, -2) if c["halves"] else pair).flatten(-2))
    return torch.cat(pieces + [x[..., at:]], -1)


def _exact_norm(s):
    c = s["case"]
    first, second = [], []
    for k in range(2):
        x, w = s["x"][k].double(), s["weight"][k].double()
        length = torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / c["d"] + EPS)
        if not c["grad"]:
            first.append(_exact_turn(s, x / length * w, False))
            continue
        g = _exact_turn(s, s["dout"][k].double(), True)
        second.append(torch.einsum("bhnd,bhnd->d", g, x / length))
        g = g * w
        along = torch.einsum("bhnd,bhnd->bhn", g, x)[..., None]
        first.append(((g - x * along / (c["d"] * length ** 2)) / length).transpose(1, 2))
    return first + second


def _exact_linear(s):
    c = s["case"]
    heads = lambda y, H: y.unflatten(2, (H, -1)).transpose(1, 2) if H else y
    x, w = _rows(s["x"]).double(), s["weight"].double()
    if not c["grad"]:
        z = torch.nn.functional.linear(x, w, s["bias"].double() if c["bias"] else None)
        if c["act"] == "silu":
            y = z * torch.sigmoid(z)
        elif c["act"]:
            y = torch.nn.functional.gelu(z, approximate="tanh" if c["act"] == "gelu_tanh" else "none")
        else:
            y = z
        if c["residual"]:
            y = y + _rows(s["residual"]).double()
        y = heads(y, c["out_heads"])
        return (y, heads(z, c["out_heads"])) if c["pre"] else y
    dz = _rows(s["dout"]).double()
    if c["act"]:
        z = _rows(s["pre"]).double().requires_grad_(True)
        with torch.enable_grad():
            f = z * torch.sigmoid(z) if c["act"] == "silu" else torch.nn.functional.gelu(
                z, approximate="tanh" if c["act"] == "gelu_tanh" else "none")
            dz, = torch.autograd.grad(f, z, dz)
    grads = [heads(torch.einsum("bnm,mk->bnk", dz, w), c["in_heads"]), torch.einsum("bnm,bnk->mk", dz, x)]
    return grads + ([dz.sum((0, 1))] if c["bias"] else [])


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] == "norm_rope" else _exact_linear(s)
