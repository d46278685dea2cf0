"""A prompt's layer beside its attention, measured: products of many rows with Q4_0 weights and an epilogue, the gated product
of a feed-forward block, the norms around a block, and rotary positions of one or several axes.

A Q4_0 block holds 32 weights: a binary16 scale d and 16 bytes, byte j with element j in its low and element j + 16 in its high
nibble.  In these products a weight is the binary16 value f16((q - 8) * d), as an element of the 8-bit cache is f16(code * d).

  gemm    y = f16(residual + scale * act(W x + bias))
  gated   y = f16(act(Wg x + bg) * (Wu x + bu))
  norm    t = residual + scale * gate * u, with u the block's output or its norm times a weight;  z = f16(norm(t) * weight + bias)
  rope    a head's pair (a, b) of row r becomes (a cos - b sin, a sin + b cos) at the angle position[axis of the pair][r] * frequency

norm(v) is v / sqrt(mean(v^2) + eps), or (v - mean) / sqrt(var + eps).  Sizes are a case's own, values come from the seed.
"""
import math

import torch

own = False

EPS = 1e-5
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
TYPES = {"f32": torch.float32, "f16": torch.float16}


def listed():
    gemm = dict(op="gemm", bias=False, act="none", scale=1.0, residual="", wide=0)
    gated = dict(op="gated", bias=False, act="silu", wide=0)
    norm = dict(op="norm", kind="rms", post=False, gate_rows=0, scale=1.0, residual="f32", t="f32", block="f16", bias=False)
    rope = dict(op="rope", heads=40, head_dim=128, rot=128, axes=1, halves=True, x="f16", y="f16", places="batch", far=4096, wide=0)
    return [
        # one token's output projection onto its residual: latency
        dict(gemm, name="out_1", rows=1, n=4096, k=4096, residual="f16"),
        # a step of 33 users: the merged q | k | v rows, with biases
        dict(gemm, name="qkv_33", rows=33, n=6144, k=4096, bias=True),
        # a ragged chunk against odd sizes: rows of an odd number of blocks, a classifier's 4099 outputs, the chunk inside wider rows
        dict(gemm, name="odd_1000", rows=1000, n=4099, k=4128, bias=True, act="gelu", wide=64),
        # a prompt's down projection with a scaled residual
        dict(gemm, name="down_2048", rows=2048, n=4096, k=14336, residual="f32", scale=0.5),
        # one token, then a step of 16 users through the gated block
        dict(gated, name="gated_1", rows=1, n=14336, k=4096),
        dict(gated, name="gated_16", rows=16, n=14336, k=4096, bias=True),
        # a short prompt of the 70B-shaped block, and the 8B-shaped block over a long one: the largest product
        dict(gated, name="gated_300", rows=300, n=28672, k=8192, act="gelu_tanh"),
        dict(gated, name="gated_2048", rows=2048, n=14336, k=4096),
        # the norm between two blocks of a step of 16 users
        dict(norm, name="norm_16", rows=16, n=4096),
        # norms after and before a block, gates that differ by sequence, a long chunk
        dict(norm, name="norm_2048", rows=2048, n=8192, post=True, gate_rows=512, scale=0.25, bias=True),
        # queries and keys of a step of 16 users, out of the fp32 rows of the projections, at the batch's positions
        dict(rope, name="rope_16", rows=16, x="f32", wide=1024),
        # an image or video prompt: three axes
        dict(rope, name="rope_4096", rows=4096, axes=3, places="given", far=100000),
    ]


def work(case):
    op, rows = case["op"], case["rows"]
    if op in ("gemm", "gated"):
        n, k, m = case["n"], case["k"], 1 if op == "gemm" else 2
        more = rows * n * (0 if op == "gated" or not case["residual"] else TYPES[case["residual"]].itemsize)
        return {"bytes": m * n * k // 32 * 18 + 2 * rows * k + 2 * rows * n + more + 4 * m * n * case["bias"], "flops": 2 * m * rows * n * k}
    if op == "norm":
        n = case["n"]
        gates = -(-rows // case["gate_rows"]) if case["gate_rows"] else 0
        each = TYPES[case["block"]].itemsize + 2 + sum(TYPES[case[b]].itemsize for b in ("residual", "t") if case[b])
        return {"bytes": rows * n * each + 4 * n * (1 + case["post"] + 2 * case["bias"] + gates), "flops": rows * n * (10 + 4 * case["post"])}
    each = case["heads"] * case["head_dim"] * (TYPES[case["x"]].itemsize + TYPES[case["y"]].itemsize) + 4 * case["axes"]
    return {"bytes": rows * each, "flops": rows * case["heads"] * case["rot"] * 4}


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.7e12 + w["flops"] / 1.9e15


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["gemm", "gemm", "gated", "gated", "norm", "rope"])
        case = dict(op=op, rows=_between(rng, 1, 4096))
        if op in ("gemm", "gated"):
            case.update(n=_between(rng, 64, 28672), k=32 * _between(rng, 4, 896), bias=rng.random() < 0.5, wide=rng.choice([0, 0, 8, 1000]))
            if rng.random() < 0.7:    # most rows are whole numbers of 256 weights
                case["k"] = max(256, case["k"] // 256 * 256)
            case["act"] = rng.choice(ACTS) if op == "gemm" else rng.choice(ACTS[1:])
            if op == "gemm":
                case.update(scale=rng.choice([1.0, 0.25]), residual=rng.choice(["", "f16", "f32"]))
        elif op == "norm":
            case.update(n=_between(rng, 32, 16384), kind=rng.choice(["rms", "layer"]), post=rng.random() < 0.5, gate_rows=rng.choice([0, 1, case["rows"], 1 + case["rows"] // 3]),
                        scale=rng.choice([1.0, 0.25]), residual=rng.choice(["", "f16", "f32"]), t=rng.choice(["", "f16", "f32"]), block=rng.choice(["f16", "f32"]),
                        bias=rng.random() < 0.3)
        else:
            head_dim = rng.choice([64, 80, 128, 192, 256])
            case.update(heads=rng.choice([1, 5, 8, 40, 72]), head_dim=head_dim, rot=rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4 * 2 - 2]), axes=rng.choice([1, 1, 2, 3, 4]),
                        halves=rng.random() < 0.5, x=rng.choice(["f16", "f32"]), y=rng.choice(["f16", "f32"]), far=_between(rng, 100, 2000000), wide=rng.choice([0, 1024]))
            case["places"] = "batch" if case["axes"] == 1 and rng.random() < 0.5 else "given"
        if _cost(case) <= most:
            return case


def _q4(n, k, gen, dev):
    """Q4_0 rows [n][k / 32][18] of weights as a trained matrix has them: normal, with a spread of its own for every row."""
    out = torch.empty((n, k // 32, 18), dtype=torch.uint8, device=dev)
    for a in range(0, n, 4096):
        m = min(4096, n - a)
        w = torch.randn((m, k // 32, 32), generator=gen, device=dev) * (torch.rand((m, 1, 1), generator=gen, device=dev) + 0.5) / math.sqrt(k)
        d = (w.gather(-1, w.abs().argmax(-1, keepdim=True)) / -8).half()
        q = torch.where(d == 0, 8.0, torch.floor(w / torch.where(d == 0, 1.0, d.float()) + 8.5)).clamp(0, 15).to(torch.uint8)
        out[a:a + m, :, :2] = d.view(torch.uint8)
        out[a:a + m, :, 2:] = q[..., :16] | (q[..., 16:] << 4)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + 29)
    op, rows = case["op"], case["rows"]
    st = dict(case=case)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if op in ("gemm", "gated"):
        n, k = case["n"], case["k"]
        st["w"] = [_q4(n, k, gen, dev) for _ in range(1 if op == "gemm" else 2)]
        st["x"] = normal(rows, k + case["wide"]).half()
        st["biases"] = [normal(n) * 0.5 for _ in st["w"]] if case["bias"] else [None] * len(st["w"])
        st["ld"] = -(-n // 8) * 8
        st["y"] = torch.zeros((rows, st["ld"]), dtype=torch.float16, device=dev)
        if op == "gemm":
            st["residual"] = normal(rows, n).to(TYPES[case["residual"]]) if case["residual"] else None
    elif op == "norm":
        n = case["n"]
        st["block"] = (normal(rows, n) * 3).to(TYPES[case["block"]])
        st["residual"] = (normal(rows, n) + 0.1).to(TYPES[case["residual"]]) if case["residual"] else None
        st["t"] = torch.zeros((rows, n), dtype=TYPES[case["t"]], device=dev) if case["t"] else None
        st["z"] = torch.zeros((rows, n), dtype=torch.float16, device=dev)
        st["weight"] = normal(n) * 0.1 + 1
        st["post"] = normal(n) * 0.1 + 1 if case["post"] else None
        st["gate"] = normal(-(-rows // case["gate_rows"]), n) if case["gate_rows"] else None
        st["bias"] = normal(n) * 0.1 if case["bias"] else None
        st["post_bias"] = normal(n) * 0.1 if case["bias"] and case["post"] else None
    else:
        pairs, axes = case["rot"] // 2, case["axes"]
        st["freqs"] = [10000.0 ** (-i / pairs) for i in range(pairs)]
        st["axis"] = [min(axes - 1, i * axes // pairs) for i in range(pairs)]    # a run of pairs for each axis
        st["table"] = torch.tensor([st["freqs"], st["axis"]], dtype=torch.float64, device=dev)
        st["x"] = normal(rows, case["heads"] * case["head_dim"] + case["wide"]).to(TYPES[case["x"]])
        st["y"] = torch.zeros((rows, case["heads"] * case["head_dim"]), dtype=TYPES[case["y"]], device=dev)
        if case["places"] == "given":
            st["places"] = torch.randint(0, case["far"], (axes, rows), generator=gen, device=dev, dtype=torch.int32)
        else:    # a sequence for every seventh row (or every row of a short step), each at its own length
            each = 7 if rows > 64 else 1
            starts = torch.arange(0, rows + each, each, device=dev).clamp(max=rows).to(torch.int32)
            new = starts[1:] - starts[:-1]
            st["starts"], st["lens"] = starts, (new + torch.randint(0, case["far"], new.shape, generator=gen, device=dev)).to(torch.int32)
    if own:
        import weight_streaming_q4_gb300 as q4
        act = dict(none=q4.Q4_ACT_NONE, relu=q4.Q4_ACT_RELU, silu=q4.Q4_ACT_SILU, gelu=q4.Q4_ACT_GELU, gelu_tanh=q4.Q4_ACT_GELU_TANH)
        kinds = {"f32": q4.Q4_TYPE_F32, "f16": q4.Q4_TYPE_F16, "": q4.Q4_TYPE_F16}
        st["kinds"] = kinds
        if op == "gemm":
            st["ep"] = q4.Epilogue.of(n, rows, act[case["act"]], case["scale"], st["biases"][0], st["residual"], kinds[case["residual"]], n)
        elif op == "gated":
            st["ep"] = q4.GatedEpilogue.of(n, act[case["act"]], *st["biases"])
        elif op == "norm":
            st["norm"] = q4.BlockNorm.of(n, q4.Q4_NORM_RMS if case["kind"] == "rms" else q4.Q4_NORM_LAYER, EPS, st["weight"], st["bias"], st["post"], st["post_bias"],
                                         case["scale"], st["gate"], n, case["gate_rows"])
        else:
            st["rope"] = q4.Rope.of(case["head_dim"], st["freqs"], st["axis"], q4.Q4_ROPE_HALVES if case["halves"] else q4.Q4_ROPE_ADJACENT)
            if case["places"] == "given":
                st["at"] = q4.RopePlaces.of(st["places"], axes, rows)
            else:
                st["at"] = q4.RopePlaces.of_batch(st["starts"], st["lens"], len(st["starts"]) - 1, rows)
    return st


def _weights(w, n, k):
    """fp32 [n][k] of Q4_0 rows; code times scale has 15 bits, so the one rounding is the one to binary16."""
    d = w[..., :2].contiguous().view(torch.float16).float()
    q = torch.cat([w[..., 2:] & 15, w[..., 2:] >> 4], dim=-1).float() - 8
    return (q * d).half().float().view(n, k)


def _act(t, act):
    if act == "relu":
        return torch.where(t > 0, t, 0.0)
    if act == "silu":
        return t / (1 + torch.exp(-t))
    if act == "gelu":
        return t * 0.5 * (1 + torch.erf(t * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return t * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t * t * t)))
    return t


def _plain_product(st, i):
    case = st["case"]
    t = st["x"][:, :case["k"]].float() @ _weights(st["w"][i], case["n"], case["k"]).T
    return t if st["biases"][i] is None else t + st["biases"][i]


def _plain_norm(v, kind, weight, bias):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * weight
    return v if bias is None else v + bias


def _row_places(st):
    """int64 [axes][rows]: the positions of every row."""
    case = st["case"]
    if case["places"] == "given":
        return st["places"].long()
    row = torch.arange(case["rows"], device=st["starts"].device)
    seq = torch.searchsorted(st["starts"].long(), row, right=True) - 1
    return (st["lens"].long()[seq] - st["starts"].long()[seq + 1] + row)[None]


def _pair_views(x, case):
    """The two members of every pair, as views [rows][heads][pairs]."""
    h = x[:, :case["heads"] * case["head_dim"]].unflatten(-1, (case["heads"], case["head_dim"]))[..., :case["rot"]]
    return (h[..., :case["rot"] // 2], h[..., case["rot"] // 2:]) if case["halves"] else (h[..., ::2], h[..., 1::2])


def run(st):
    case, op = st["case"], st["case"]["op"]
    if own:
        import weight_streaming_q4_gb300 as q4
        rows, kinds = case["rows"], st["kinds"]
        if op == "gemm":
            q4.q4_gemm(st["w"][0], st["x"], case["k"] + case["wide"], case["n"], case["k"], rows, st["ep"], st["y"], st["ld"])
            return st["y"]
        if op == "gated":
            q4.q4_gemm_gated(*st["w"], st["x"], case["k"] + case["wide"], case["n"], case["k"], rows, st["ep"], st["y"], st["ld"])
            return st["y"]
        if op == "norm":
            n = case["n"]
            q4.q4_block_norm(st["norm"], rows, st["block"], kinds[case["block"]], n, st["residual"], kinds[case["residual"]], n, st["t"], kinds[case["t"]], n,
                             st["z"], q4.Q4_TYPE_F16, n)
            return [st["z"]] + ([st["t"]] if case["t"] else [])
        x, y = st["x"], st["y"]
        q4.q4_rope(st["rope"], st["at"], case["heads"], x, kinds[case["x"]], x.shape[1], y, kinds[case["y"]], y.shape[1])
        return y
    if op == "gemm":
        t = _act(_plain_product(st, 0), case["act"]) * case["scale"]
        st["y"][:, :case["n"]] = (t if st["residual"] is None else t + st["residual"].float()).half()
        return st["y"]
    if op == "gated":
        st["y"][:, :case["n"]] = (_act(_plain_product(st, 0), case["act"]) * _plain_product(st, 1)).half()
        return st["y"]
    if op == "norm":
        u = st["block"].float()
        if case["post"]:
            u = _plain_norm(u, case["kind"], st["post"], st["post_bias"])
        u = u * case["scale"]
        if case["gate_rows"]:
            u = u * st["gate"].repeat_interleave(case["gate_rows"], 0)[:case["rows"]]
        t = u if st["residual"] is None else u + st["residual"].float()
        st["z"].copy_(_plain_norm(t, case["kind"], st["weight"], st["bias"]))
        if case["t"]:
            st["t"].copy_(t)
        return [st["z"]] + ([st["t"]] if case["t"] else [])
    angle = _row_places(st)[st["table"][1].long()].T * st["table"][0]    # angles of far positions, in 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    y = st["y"].copy_(st["x"][:, :st["y"].shape[1]])
    (a, b), (c, d) = _pair_views(st["x"], case), _pair_views(y, case)
    a, b = a.float(), b.float()
    c.copy_(a * cos - b * sin)
    d.copy_(a * sin + b * cos)
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op, rows = case["op"], case["rows"]
    if op in ("gemm", "gated"):
        n, k = case["n"], case["k"]

        def product(i):
            parts = []
            for a in range(0, n, 2048):
                blocks = st["w"][i][a:a + 2048]
                scale = (blocks[:, :, 0].to(torch.int16) + blocks[:, :, 1].to(torch.int16) * 256).view(torch.float16).double()
                codes = torch.stack([blocks[:, :, 2:] % 16, blocks[:, :, 2:] // 16], dim=2).flatten(2).double() - 8
                parts.append((codes * scale[:, :, None]).half().double().reshape(-1, k))    # a weight as these products take it
            t = torch.cat([st["x"][:, :k].double() @ p.T for p in parts], dim=1)
            return t + st["biases"][i].double() if case["bias"] else t

        f = {"none": lambda t: t, "relu": lambda t: t.clamp(min=0), "silu": lambda t: t * torch.sigmoid(t), "gelu": torch.nn.functional.gelu,
             "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[case["act"]]
        t = f(product(0))
        if op == "gated":
            t = t * product(1)
        else:
            t = t * case["scale"]
            if st["residual"] is not None:
                t = t + st["residual"].double()
        out = torch.zeros((rows, st["ld"]), dtype=torch.float64, device=t.device)
        out[:, :n] = t
        return out
    if op == "norm":
        def normed(v, weight, bias):
            off = v.mean(-1, keepdim=True) if case["kind"] == "layer" else torch.zeros_like(v[:, :1])
            spread = ((v - off) ** 2).mean(-1, keepdim=True)
            return (v - off) * torch.rsqrt(spread + EPS) * weight.double() + (0 if bias is None else bias.double())

        u = st["block"].double()
        u = normed(u, st["post"], st["post_bias"]) if case["post"] else u
        if case["gate_rows"]:
            u = u * st["gate"].double()[torch.arange(rows, device=u.device) // case["gate_rows"]]
        t = u * case["scale"] + (0 if st["residual"] is None else st["residual"].double())
        return [normed(t, st["weight"], st["bias"])] + ([t] if case["t"] else [])
    x = st["x"].double()
    y = x[:, :st["y"].shape[1]].clone()
    if case["places"] == "given":
        places = st["places"].double()
    else:
        starts, lens = st["starts"].tolist(), st["lens"].tolist()
        places = torch.tensor([[n - (b - a) + i for a, b, n in zip(starts, starts[1:], lens) for i in range(b - a)]], dtype=torch.float64, device=x.device)
    half, hd = case["rot"] // 2, case["head_dim"]
    for i, (freq, axis) in enumerate(zip(st["freqs"], st["axis"])):
        turn = torch.polar(torch.ones_like(places[axis]), places[axis] * freq)[:, None]
        first = i if case["halves"] else 2 * i
        at = torch.arange(case["heads"], device=x.device) * hd + first
        to = at + (half if case["halves"] else 1)
        z = torch.complex(x[:, at], x[:, to]) * turn
        y[:, at], y[:, to] = z.real, z.imag
    return y
