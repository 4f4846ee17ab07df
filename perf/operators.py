"""Measured cases of the operators around block-sparse attention: the position
rotation over several axes, the block selection that makes an attention mask,
attention over the selected blocks, and a training step (forward and backward)
of block-sparse attention.

``run`` computes a case in elementary torch operations where ``own`` is false,
and calls the library where it is true.  Inputs are bf16 ``[B, H, N, d]`` unless
a case says otherwise; a rotation reads the projections' ``[B, N, H, d]``.
"""
import math

import torch

own = False

LOG2_LIMIT = 31   # elements of one dense score matrix that the plain forms hold at a time


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a tiny latent video, every token of one small layer: latency counts
        {"name": "rope_tiny", "op": "rope", "B": 1, "H": 2, "F": 4, "h": 16, "w": 16, "text": 0, "d": 64,
         "at": 16, "ah": 24, "aw": 24, "halves": False, "inverse": False, "dtype": "bf16"},
        # Q and K of one 480p layer (21 frames of 30 x 52 latents), token-major projections in,
        # the attention's head-major layout out
        {"name": "rope_480p", "op": "rope", "B": 1, "H": 24, "F": 21, "h": 30, "w": 52, "text": 0, "d": 128,
         "at": 44, "ah": 42, "aw": 42, "halves": False, "inverse": False, "dtype": "bf16"},
        # the gradients of a 720p layer's rotation on their way back to the projections
        {"name": "rope_720p_backward", "op": "rope", "B": 1, "H": 24, "F": 21, "h": 45, "w": 80, "text": 0,
         "d": 128, "at": 32, "ah": 48, "aw": 48, "halves": True, "inverse": True, "dtype": "bf16"},
        # text tokens before the latents: explicit positions, an odd token count, fp32
        {"name": "rope_text_fp32", "op": "rope", "B": 2, "H": 5, "F": 3, "h": 33, "w": 41, "text": 37, "d": 64,
         "at": 16, "ah": 16, "aw": 16, "halves": False, "inverse": False, "dtype": "fp32"},
        # block selection alone: a tiny layer, then the 480p and 720p layers
        {"name": "select_tiny", "op": "select", "B": 1, "H": 2, "N": 1024, "d": 64, "bq": 64, "bk": 64, "keep": 5,
         "first": 0, "diagonal": True},
        {"name": "select_480p", "op": "select", "B": 1, "H": 24, "N": 32760, "d": 128, "bq": 64, "bk": 64,
         "keep": 103, "first": 1, "diagonal": True},
        {"name": "select_720p", "op": "select", "B": 1, "H": 24, "N": 75600, "d": 128, "bq": 128, "bk": 128,
         "keep": 89, "first": 0, "diagonal": True},
        # a request's attention with its own mask: select, plan, attend
        {"name": "attend_odd", "op": "attend", "B": 2, "H": 3, "N": 5003, "d": 64, "bq": 32, "bk": 64, "keep": 17,
         "first": 2, "diagonal": False},
        {"name": "attend_480p", "op": "attend", "B": 1, "H": 24, "N": 32760, "d": 128, "bq": 64, "bk": 64,
         "keep": 103, "first": 1, "diagonal": True},
        # one training step of the attention: forward, then the gradients of Q, K and V
        {"name": "train_tiny", "op": "train", "B": 1, "H": 2, "N": 1024, "d": 64, "bq": 64, "bk": 64,
         "density": 0.3, "segments": False},
        {"name": "train_segments", "op": "train", "B": 1, "H": 5, "N": 6007, "d": 128, "bq": 16, "bk": 200,
         "density": 0.4, "segments": True},
        {"name": "train_480p", "op": "train", "B": 1, "H": 24, "N": 32760, "d": 128, "bq": 64, "bk": 64,
         "density": 0.25, "segments": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["rope", "select", "attend", "train"])
    d = rng.choice([64, 128])
    B = rng.choice([1, 1, 1, 2])
    if op == "rope":
        half = d // 2
        ah = 2 * rng.randint(1, half // 2)
        aw = 2 * rng.randint(1, half // 2)
        at = rng.choice([d - ah - aw, 2 * rng.randint(1, (d - ah - aw) // 2)])
        F, h, w = _log_int(rng, 1, 21), _log_int(rng, 1, 45), _log_int(rng, 1, 80)
        return {"op": op, "B": B, "H": rng.randint(1, 12), "F": F, "h": h, "w": w,
                "text": rng.choice([0, 0, rng.randint(1, 300)]), "d": d, "at": at, "ah": ah, "aw": aw,
                "halves": rng.random() < 0.5, "inverse": rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    if op == "select":
        N, bq, bk = _log_int(rng, 1, 75600), rng.choice([32, 48, 64, 128]), rng.choice([32, 64, 80, 128])
        n = -(-N // bk)
        return {"op": op, "B": B, "H": rng.randint(1, 12), "N": N, "d": d, "bq": bq, "bk": bk,
                "keep": rng.randint(1, max(1, n // 2)), "first": rng.choice([0, 0, 1, 3]),
                "diagonal": rng.random() < 0.5}
    if op == "attend":
        N, bq, bk = _log_int(rng, 64, 20000), rng.choice([32, 64, 128]), rng.choice([32, 64, 128])
        n = -(-N // bk)
        return {"op": op, "B": B, "H": rng.randint(1, 8), "N": N, "d": d, "bq": bq, "bk": bk,
                "keep": rng.randint(1, max(1, n // 3)), "first": rng.choice([0, 1, 2]),
                "diagonal": rng.random() < 0.5}
    N, segments = _log_int(rng, 64, 16000), rng.random() < 0.3
    return {"op": op, "B": B, "H": rng.randint(1, 8), "N": N, "d": d,
            "bq": 16 if segments else rng.choice([32, 64, 128]),
            "bk": rng.randint(64, 300) if segments else rng.choice([32, 64, 128, 256]),
            "density": round(rng.uniform(0.05, 0.6), 3), "segments": segments}


# ------------------------------------------------------------------ the inputs
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _cdiv(a, b):
    return -(-a // b)


def _features(g, B, H, N, d):
    """Tokens that resemble their neighbours, as latents of one video do: white
    noise over a component that changes every 40 tokens."""
    slow = torch.randn((B, H, _cdiv(N, 40), d), generator=g, device="cuda")
    x = torch.randn((B, H, N, d), generator=g, device="cuda")
    return x.add_(slow.repeat_interleave(40, dim=2)[:, :, :N], alpha=0.7).to(torch.bfloat16)


def _segment_bounds(g, N, lo, hi):
    """Ascending bounds 0 .. N of segments of lo to hi tokens."""
    steps = torch.randint(lo, hi + 1, (N // lo + 1,), generator=g, device="cuda")
    cuts = torch.cumsum(steps, 0)
    cuts = cuts[cuts <= N - lo]
    ends = torch.tensor([0, N], device="cuda")
    return torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)


def _blocks(g, B, H, nq, nk, density):
    """Banded-plus-random block mask: denser near the diagonal, the diagonal on,
    one whole row and one whole column of blocks off where there are many."""
    i = (torch.arange(nq, device="cuda") + 0.5) / nq
    j = (torch.arange(nk, device="cuda") + 0.5) / nk
    away = (i[:, None] - j[None, :]).abs() * max(nq, nk)
    w = 1 + 4 * torch.exp(-away / 16)
    p = (w * (density / w.mean())).clamp(max=1)
    on = torch.rand((B, H, nq, nk), generator=g, device="cuda") < p
    on |= away < 0.5 * max(1.0, max(nq, nk) / min(nq, nk))
    if nq > 8 and nk > 8:
        on[:, :, nq // 3] = False
        on[:, :, :, nk // 2] = False
    return on.to(torch.uint8).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = case
    s = {"case": case}
    if c["op"] == "rope":
        grid = (c["F"], c["h"], c["w"])
        n = c["text"] + c["F"] * c["h"] * c["w"]
        dt = DTYPES[c["dtype"]]
        shape = (c["B"], c["H"], n, c["d"]) if c["inverse"] else (c["B"], n, c["H"], c["d"])
        s["x"] = [torch.randn(shape, generator=g, device="cuda").to(dt) for _ in range(2)]
        s["positions"] = None
        if c["text"]:
            # text tokens run along the time axis before the latents, as far out as their prompt starts
            t = torch.arange(c["F"] * c["h"] * c["w"], device="cuda")
            video = torch.stack([t // (c["h"] * c["w"]) + c["text"], t // c["w"] % c["h"], t % c["w"]], 1)
            start = torch.randint(0, 100000, (1,), generator=g, device="cuda")
            text = (torch.arange(c["text"], device="cuda") + start)[:, None].expand(-1, 3)
            s["positions"] = torch.cat([text, video]).to(torch.int32).contiguous()
        s["grid"] = grid
        return s
    B, H, N, d = c["B"], c["H"], c["N"], c["d"]
    s["q"], s["k"] = _features(g, B, H, N, d), _features(g, B, H, N, d)
    if c["op"] == "select":
        return s
    s["v"] = torch.randn((B, H, N, d), generator=g, device="cuda").to(torch.bfloat16)
    if c["op"] == "train":
        s["dout"] = torch.randn((B, H, N, d), generator=g, device="cuda").to(torch.bfloat16)
        if c["segments"]:
            s["q_bounds"] = _segment_bounds(g, N, c["bq"], c["bk"])
            s["k_bounds"] = _segment_bounds(g, N, c["bq"], c["bk"])
            nq, nk = s["q_bounds"].numel() - 1, s["k_bounds"].numel() - 1
        else:
            nq, nk = _cdiv(N, c["bq"]), _cdiv(N, c["bk"])
        s["blocks"] = _blocks(g, B, H, nq, nk, c["density"])
    if own:
        # what a program keeps from step to step: the plans (their storage, for a mask that changes)
        import block_sparse_attention_tsr_gb300 as tsr
        if c["op"] == "train":
            mask = _mask(s)
            s["plan"], s["plan_backward"] = tsr.tsr_plan(mask), tsr.tsr_backward_plan(mask)
        else:
            s["plan"] = tsr.tsr_plan(tsr.make_mask(tsr.UNIFORM, B, H, N, d, bq=c["bq"], bk=c["bk"],
                                                   blocks=_select_own(s)))
    return s


# --------------------------------------------------------- the library's calls
def _mask(s):
    import block_sparse_attention_tsr_gb300 as tsr
    c = s["case"]
    shape = (c["B"], c["H"], c["N"], c["d"])
    if c["segments"]:
        return tsr.make_mask(tsr.SEGMENTS, *shape, q_bounds=s["q_bounds"], k_bounds=s["k_bounds"],
                             blocks=s["blocks"])
    return tsr.make_mask(tsr.UNIFORM, *shape, bq=c["bq"], bk=c["bk"], blocks=s["blocks"])


def _rope_own(s):
    import block_sparse_attention_tsr_gb300 as tsr
    c = s["case"]
    kw = dict(axis_dims=(c["at"], c["ah"], c["aw"]), theta=10000.0, halves=c["halves"])
    if s["positions"] is not None:
        kw["positions"] = s["positions"]
    else:
        kw["grid"] = s["grid"]
    if c["inverse"]:
        # head-major gradients in, the projections' token-major gradients out
        out = [torch.empty((c["B"], x.shape[2], c["H"], c["d"]), dtype=x.dtype, device=x.device) for x in s["x"]]
        tsr.tsr_rope_backward(s["x"], out=[o.transpose(1, 2) for o in out], **kw)
        return out
    return tsr.tsr_rope([x.transpose(1, 2) for x in s["x"]], **kw)


def _select_own(s):
    import block_sparse_attention_tsr_gb300 as tsr
    c = s["case"]
    return tsr.tsr_block_select(s["q"], s["k"], c["keep"], bq=c["bq"], bk=c["bk"], first=c["first"],
                                diagonal=c["diagonal"])


def _attend_own(s):
    import block_sparse_attention_tsr_gb300 as tsr
    c = s["case"]
    blocks = _select_own(s)
    s["plan"].update(tsr.make_mask(tsr.UNIFORM, c["B"], c["H"], c["N"], c["d"], bq=c["bq"], bk=c["bk"],
                                   blocks=blocks))
    out, lse = tsr.tsr_bsa_forward(s["q"], s["k"], s["v"], s["plan"])
    return blocks, out, lse


def _train_own(s):
    import block_sparse_attention_tsr_gb300 as tsr
    out, lse = tsr.tsr_bsa_forward(s["q"], s["k"], s["v"], s["plan"])
    dq, dk, dv = tsr.tsr_bsa_backward(s["q"], s["k"], s["v"], out, lse, s["dout"], s["plan_backward"])
    return out, lse, dq, dk, dv


# -------------------------------------------------------------- the plain forms
def _angles(s, dtype):
    """Angles [N, rotated channels / 2]: position x frequency in 64 bits, so that
    far positions keep their place on the circle."""
    c = s["case"]
    pos = s["positions"]
    if pos is None:
        F, h, w = s["grid"]
        t = torch.arange(F * h * w, device="cuda")
        pos = torch.stack([t // (h * w), t // w % h, t % w], 1)
    parts = []
    for axis, width in enumerate((c["at"], c["ah"], c["aw"])):
        j = torch.arange(width // 2, device="cuda", dtype=torch.float64)
        parts.append(pos[:, axis, None].double() * 10000.0 ** (-2 * j / width))
    a = torch.cat(parts, 1)
    if c["inverse"]:
        a = -a
    return torch.cos(a).to(dtype), torch.sin(a).to(dtype)


def _pair_places(s):
    """The channels of each pair's first and second element."""
    c = s["case"]
    first, second, at = [], [], 0
    for width in (c["at"], c["ah"], c["aw"]):
        j = torch.arange(width // 2, device="cuda")
        first.append(at + (j if c["halves"] else 2 * j))
        second.append(at + (j + width // 2 if c["halves"] else 2 * j + 1))
        at += width
    return torch.cat(first), torch.cat(second)


def _rope_plain(s):
    c = s["case"]
    cos, sin = _angles(s, torch.float32)
    i, j = _pair_places(s)
    out = []
    for x in s["x"]:
        head_major = x if c["inverse"] else x.transpose(1, 2)
        y = head_major.float().contiguous()
        a, b = y[..., i], y[..., j]
        y[..., i] = a * cos - b * sin
        y[..., j] = a * sin + b * cos
        y = y.to(x.dtype)
        out.append(y.transpose(1, 2).contiguous() if c["inverse"] else y)
    return out


def _means(x, b):
    """Block means [B, H, ceil(N / b), d] in 64 bits; the last block's over its own rows."""
    B, H, N, d = x.shape
    n = _cdiv(N, b)
    y = torch.zeros((B, H, n * b, d), dtype=torch.float64, device=x.device)
    y[:, :, :N] = x
    rows = torch.full((n, 1), float(b), dtype=torch.float64, device=x.device)
    rows[-1] = N - (n - 1) * b
    return y.view(B, H, n, b, d).sum(3) / rows


def _select_plain(s):
    c = s["case"]
    N, bq, bk = c["N"], c["bq"], c["bk"]
    # 64 bits: whether a block is kept turns on scores next to the last one kept
    score = _means(s["q"], bq) @ _means(s["k"], bk).transpose(-1, -2)
    nq, nk = score.shape[-2:]
    i, j = torch.arange(nq, device="cuda")[:, None], torch.arange(nk, device="cuda")[None, :]
    forced = (j < c["first"]).expand(nq, nk)
    if c["diagonal"]:
        last = torch.clamp((i + 1) * bq, max=N) - 1
        forced = forced | ((j * bk <= last) & ((j + 1) * bk > i * bq))
    score = torch.where(forced, math.inf, score)
    order = torch.argsort(score, dim=-1, descending=True, stable=True)
    kept = torch.zeros((c["B"], c["H"], nq, nk), dtype=torch.uint8, device="cuda")
    kept.scatter_(-1, order[..., : c["keep"]], 1)
    return kept | forced.to(torch.uint8)


def _allowed(s, blocks):
    """Element mask of a block mask's heads, [heads, N, N]."""
    c = s["case"]
    t = torch.arange(c["N"], device="cuda", dtype=torch.int32)
    if c.get("segments"):
        i = torch.bucketize(t, s["q_bounds"][1:], right=True)
        j = torch.bucketize(t, s["k_bounds"][1:], right=True)
    else:
        i, j = (t // c["bq"]).long(), (t // c["bk"]).long()
    return blocks[:, i][:, :, j].bool()


def _probabilities(s, q, k, blocks):
    """P and lse of some heads: the masked softmax, rows with nothing allowed all zero."""
    x = torch.bmm(q, k.transpose(1, 2)).mul_(1 / math.sqrt(q.shape[-1]))
    x.masked_fill_(~_allowed(s, blocks), -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    return x.div_(torch.where(total == 0, 1.0, total)), lse


def _by_heads(s, one, *tensors):
    """`one` over as many (batch, head) pairs at a time as keep a dense score matrix in memory."""
    c = s["case"]
    heads = [t.flatten(0, 1) for t in tensors]
    step = max(1, 2 ** LOG2_LIMIT // (c["N"] * c["N"]))
    parts = [one(*(t[i:i + step] for t in heads)) for i in range(0, c["B"] * c["H"], step)]
    return [torch.cat(p).view(c["B"], c["H"], *p[0].shape[1:]) for p in zip(*parts)]


def _attend_plain(s):
    blocks = _select_plain(s)

    def one(q, k, v, blk):
        p, lse = _probabilities(s, q.float(), k.float(), blk)
        return torch.bmm(p, v.float()).to(q.dtype), lse

    return [blocks] + _by_heads(s, one, s["q"], s["k"], s["v"], blocks)


def _train_plain(s):
    scale = 1 / math.sqrt(s["case"]["d"])

    def one(q, k, v, do, blk):
        dt, q, k, v, do = q.dtype, q.float(), k.float(), v.float(), do.float()
        p, lse = _probabilities(s, q, k, blk)
        o = torch.bmm(p, v)
        dv = torch.bmm(p.transpose(1, 2), do)
        dp = torch.bmm(do, v.transpose(1, 2))
        ds = p.mul_(dp.sub_((do * o).sum(-1, keepdim=True))).mul_(scale)
        return (o.to(dt), lse, torch.bmm(ds, k).to(dt), torch.bmm(ds.transpose(1, 2), q).to(dt), dv.to(dt))

    return _by_heads(s, one, s["q"], s["k"], s["v"], s["dout"], s["blocks"])


def run(state):
    op = state["case"]["op"]
    if own:
        if op == "rope":
            return _rope_own(state)
        if op == "select":
            return _select_own(state)
        return _attend_own(state) if op == "attend" else _train_own(state)
    if op == "rope":
        return _rope_plain(state)
    if op == "select":
        return _select_plain(state)
    return _attend_plain(state) if op == "attend" else _train_plain(state)


# --------------------------------------------------------------- the work
def work(case):
    c = case
    d = c["d"]
    if c["op"] == "rope":
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[c["dtype"]]
        n = c["text"] + c["F"] * c["h"] * c["w"]
        values = 2 * c["B"] * c["H"] * n
        rotated = c["at"] + c["ah"] + c["aw"]
        return {"bytes": values * d * 2 * size + (12 * n if c["text"] else 0), "flops": values * rotated * 3}
    B, H, N = c["B"], c["H"], c["N"]
    tensor = B * H * N * d * 2
    if c["op"] in ("select", "attend"):
        nq, nk = _cdiv(N, c["bq"]), _cdiv(N, c["bk"])
        select = 2 * B * H * nq * nk * d + 2 * B * H * N * d
        if c["op"] == "select":
            return {"bytes": 2 * tensor + B * H * nq * nk, "flops": select}
        pairs = B * H * N * min(N, c["keep"] * c["bk"])
        return {"bytes": 4 * tensor + B * H * (nq * nk + 4 * N), "flops": select + 4 * d * pairs}
    pairs = B * H * N * N * c["density"]
    # forward 4 d, backward 10 d a pair; Q, K, V and dO in, O, dQ, dK and dV out
    return {"bytes": 8 * tensor + 4 * B * H * N, "flops": 14 * d * pairs}


# ------------------------------------------------------- the definition, 64 bits
def _exact_rope(s):
    c = s["case"]
    if s["positions"] is None:
        F, h, w = s["grid"]
        pos = torch.cartesian_prod(*(torch.arange(n, device="cuda", dtype=torch.float64) for n in (F, h, w)))
        pos = pos.view(-1, 3)
    else:
        pos = s["positions"].double()
    turned = []
    for x in s["x"]:
        z = (x if c["inverse"] else x.transpose(1, 2)).double()
        pieces, at = [], 0
        for axis, width in enumerate((c["at"], c["ah"], c["aw"])):
            part = z[..., at:at + width]
            at += width
            pair = part.unflatten(-1, (2, width // 2)).transpose(-1, -2) if c["halves"] else part.unflatten(-1, (-1, 2))
            speed = torch.exp(torch.arange(0, width, 2, device="cuda", dtype=torch.float64) * (-math.log(10000.0) / width))
            angle = torch.outer(pos[:, axis], speed)
            turn = torch.polar(torch.ones_like(angle), -angle if c["inverse"] else angle)
            pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            pieces.append((pair.transpose(-1, -2) if c["halves"] else pair).flatten(-2))
        z = torch.cat(pieces + [z[..., at:]], -1)
        turned.append(z.transpose(1, 2) if c["inverse"] else z)
    return turned


def _exact_attention(s, blocks, head):
    """One head in 64 bits: P, O and lse from exponentials of the allowed scores."""
    b, h = divmod(head, s["case"]["H"])
    q, k, v = (s[n][b, h].double() for n in "qkv")
    ok = _allowed(s, blocks[b, h][None])[0]
    score = torch.where(ok, q @ k.mT / math.sqrt(q.shape[1]), -math.inf)
    lse = torch.logsumexp(score, 1)
    p = torch.where(ok, torch.exp(score - lse[:, None]), 0.0)
    return q, k, v, p, p @ v, lse


def exact(case, seed):
    c = case
    if c["op"] == "select":
        return None
    if c["op"] == "rope":
        return _exact_rope(prepare(case, seed))
    if c["B"] * c["H"] * c["N"] ** 2 * c["d"] > 1e12:
        return None
    s = prepare(case, seed)
    blocks = s["blocks"] if c["op"] == "train" else _select_plain(s)
    rows = []
    for head in range(c["B"] * c["H"]):
        q, k, v, p, o, lse = _exact_attention(s, blocks, head)
        if c["op"] == "attend":
            rows.append((o, lse))
            continue
        do = s["dout"][divmod(head, c["H"])].double()
        ds = p * (do @ v.mT)
        ds = (ds - p * ds.sum(1, keepdim=True)) / math.sqrt(c["d"])
        rows.append((o, lse, ds @ k, ds.mT @ q, p.mT @ do))
    outs = [torch.stack(x).view(c["B"], c["H"], *x[0].shape) for x in zip(*rows)]
    return ([None] if c["op"] == "attend" else []) + outs
