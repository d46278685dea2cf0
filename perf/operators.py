"""The paged KV cache's operators, measured: writing tokens into pages, reading them back, and attending to them.

A sequence's keys and values sit in pages of ``page`` positions, each page [kv heads][page][head_dim], as binary16 or as
Q8 (per 32 values of a head one binary16 scale d = f16(max|x| / 127) and the codes rint(x / d); an element stands for
f16(code * d)).  Row r of the new tokens belongs to sequence s when token_starts[s] <= r < token_starts[s + 1]; the last of
them stands at position kv_lens[s] - 1.  A query at position p sees position t when t <= p and, with a window W, also
t > p - W or t < sinks.

Lengths are a fixed function of the case (a low-discrepancy spread between its least and its largest ones), values come from
the seed.
"""
import math

import numpy as np
import torch

own = False

HEADS = {"8b": (32, 8, 128), "70b": (64, 8, 128), "64x8": (8, 8, 64), "256x1": (16, 1, 256), "192x4": (12, 4, 192)}
PAD = 3    # rows behind the last sequence, as in a batch padded to a captured size


def listed():
    attn = dict(op="attn", heads="8b", page=64, cache="f16", q="f32", window=0, sinks=0)
    return [
        # one user, first tokens of an answer: the smallest context bucket; launch and latency
        dict(attn, name="decode_1x512", seqs=1, new_min=1, new=1, ctx_min=511, ctx=511),
        # one user, the largest context bucket
        dict(attn, name="decode_1x4096", seqs=1, new_min=1, new=1, ctx_min=4095, ctx=4095),
        # a serving batch of 64 users at different lengths, 8-bit cache, the 70B-shaped heads
        dict(attn, name="decode_64_q8", heads="70b", cache="q8", seqs=64, new_min=1, new=1, ctx_min=200, ctx=8191),
        # long chats kept to a window and four first tokens, the pages between given back
        dict(attn, name="decode_16_window", heads="64x8", page=16, seqs=16, new_min=1, new=1, ctx_min=3000, ctx=32767, window=1024, sinks=4),
        # drafted tokens to verify: five new tokens for each of eight users
        dict(attn, name="verify_8x5_q8", page=16, cache="q8", seqs=8, new_min=5, new=5, ctx_min=1000, ctx=4091),
        # a mixed step: prompt chunks of several lengths beside single tokens
        dict(attn, name="mixed_8", q="f16", seqs=8, new_min=1, new=2049, ctx_min=0, ctx=2000),
        # a prompt's chunk of 512 over an 8-bit cache, the 70B-shaped heads
        dict(attn, name="chunk_512_q8", heads="70b", q="f16", cache="q8", seqs=1, new_min=512, new=512, ctx_min=7680, ctx=7680),
        # the last chunk of a 16k prompt: the largest product
        dict(attn, name="chunk_2048", q="f16", seqs=1, new_min=2048, new=2048, ctx_min=14336, ctx=14336),
        # a prompt chunk under a window with sinks, wide heads, one value head
        dict(attn, name="chunk_window", heads="256x1", q="f16", page=32, seqs=2, new_min=1000, new=2047, ctx_min=1, ctx=6000, window=1000, sinks=4),
        # the cache write of one step of 16 users, from the fp32 rows of the projections
        dict(op="write", name="write_16", heads="8b", page=64, cache="f16", src="f32", seqs=16, new_min=1, new=1, ctx_min=100, ctx=511),
        # prompts quantised into the cache, and read back as what the cache now holds
        dict(op="requant", name="requant_q8", heads="8b", page=64, cache="q8", src="f32", seqs=3, new_min=1001, new=8000, ctx_min=0, ctx=500),
        # an 8-bit cache of a sequence read out into the binary16 bucket of the one-sequence decoder
        dict(op="read", name="read_bucket_q8", heads="8b", page=64, cache="q8", src="f16", seqs=1, new_min=4096, new=4096, ctx_min=0, ctx=0),
    ]


def _spread(lo, hi, n, phase, power):
    """n whole lengths between lo and hi, hi first; a power above 1 makes most of them short, as prompts beside single tokens are."""
    return [lo + int((hi - lo) * (1 - (i * phase) % 1.0) ** power) for i in range(n)]


def lengths(case):
    """(new tokens, positions after them) of every sequence."""
    new = _spread(case["new_min"], case["new"], case["seqs"], 0.6180339887, 5)
    ctx = _spread(case["ctx_min"], case["ctx"], case["seqs"], 0.7548776662, 1)
    return new, [a + b for a, b in zip(new, ctx)]


def _visible(case):
    """Per sequence: (sum over its queries of the positions they see, positions that at least one of them sees)."""
    w, sinks = case.get("window", 0), case.get("sinks", 0)
    places = [np.arange(length - n, length, dtype=np.int64) for n, length in zip(*lengths(case))]
    firsts = [np.maximum(0, p - w + 1) if w else np.zeros_like(p) for p in places]
    pairs = [int(np.sum(p - f + 1 + np.minimum(f, sinks))) for p, f in zip(places, firsts)]
    seen = [int(p[-1] + 1 - f[0] + min(f[0], sinks)) for p, f in zip(places, firsts)]
    return pairs, seen


def work(case):
    n_q, n_kv, hd = HEADS[case["heads"]]
    new, _ = lengths(case)
    tokens = sum(new)
    cached = 2 * n_kv * hd * (2 if case["cache"] == "f16" else 1 + 2 / 32)    # bytes of a position's key and value
    if case["op"] == "attn":
        pairs, seen = _visible(case)
        rows = tokens * n_q * hd * ((4 if case["q"] == "f32" else 2) + 2)
        return {"bytes": rows + sum(seen) * cached, "flops": 4 * n_q * hd * sum(pairs)}
    rows = 2 * tokens * n_kv * hd * (4 if case["src"] == "f32" else 2)
    if case["op"] == "write":
        return {"bytes": rows + tokens * cached, "flops": 2 * tokens * n_kv * hd}
    if case["op"] == "read":
        return {"bytes": rows + tokens * cached, "flops": 2 * tokens * n_kv * hd}
    return {"bytes": rows + 2 * tokens * cached + 4 * tokens * n_kv * hd, "flops": 8 * tokens * n_kv * hd}


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.9e15


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        case = dict(op=rng.choice(["attn"] * 4 + ["write", "requant", "read"]), heads=rng.choice(sorted(HEADS)), page=rng.choice([16, 32, 64, 128]),
                    cache=rng.choice(["f16", "q8"]), seqs=_between(rng, 1, 64), ctx=_between(rng, 1, 32768) - 1)
        case["new"] = rng.choice([1, rng.randint(2, 16), _between(rng, 17, 4096)])
        case["new_min"] = rng.choice([1, case["new"]])
        case["ctx_min"] = rng.choice([case["ctx"] // 8, case["ctx"]])
        if case["op"] == "attn":
            case["q"] = rng.choice(["f32", "f16"])
            case["window"] = rng.choice([0, _between(rng, 16, 4096)])
            case["sinks"] = rng.choice([0, 1, 4, 37]) if case["window"] else 0
        else:
            case["src"] = rng.choice(["f32", "f16"])
            if case["op"] == "requant":
                case["cache"] = "q8"
            elif case["op"] == "write":
                case["cache"] = "f16"
            elif case["op"] == "read":
                case["new"] = case["new_min"] = _between(rng, 17, 8192)
                case["ctx"] = case["ctx_min"] = 0
            case["seqs"] = min(case["seqs"], 16)
        padded = case["seqs"] * case["new"] * HEADS[case["heads"]][0] * (case["new"] + case["ctx"])    # scores of a padded batch
        pool = case["seqs"] * (case["new"] + case["ctx"]) * HEADS[case["heads"]][1] * HEADS[case["heads"]][2]
        if _cost(case) <= most and padded <= 1.2e9 and pool <= 4e8:
            return case


def _quantise(x):
    """x [..., head_dim] -> (int8 codes, binary16 scales [..., head_dim / 32]).  32 bits are enough: 127 * d and (n + 1/2) * d fit them."""
    b = x.unflatten(-1, (-1, 32))
    d = (b.abs().amax(-1, keepdim=True) / 127.0).half()
    df = d.float()
    code = torch.where(df > 0, torch.round(b / torch.where(df > 0, df, 1.0)), 0.0).clamp(-127, 127)
    return code.to(torch.int8).flatten(-2), d.squeeze(-1)


def _values(code, d):
    """What Q8 codes stand for: f16(code * d)."""
    return (code.float().unflatten(-1, (-1, 32)) * d.float().unsqueeze(-1)).flatten(-2).half()


def prepare(case, seed):
    dev = torch.device("cuda")
    n_q, n_kv, hd = HEADS[case["heads"]]
    page, q8 = case["page"], case["cache"] == "q8"
    new, total = lengths(case)
    tokens, rows = sum(new), sum(new) + PAD
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + 17)
    width = max(-(-t // page) for t in total) + 1
    used = [-(-t // page) for t in total]
    n_pages = sum(used) + 2
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32).cpu().numpy()
    table = np.full((len(new), width), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = order[at:at + n]
        at += n
    if case.get("window"):    # pages that no query sees any more were given back
        for s, (n, t) in enumerate(zip(new, total)):
            lo, hi = -(-case["sinks"] // page), max(0, t - n - case["window"] + 1) // page
            table[s, lo:max(lo, hi)] = -1
    st = dict(case=case, rows=rows, new=max(new), longest=max(total), n_pages=n_pages, n_q=n_q, n_kv=n_kv, hd=hd, page=page, q8=q8, width=width,
              table=torch.from_numpy(table).to(dev), starts=torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=dev),
              lens=torch.tensor(total, dtype=torch.int32, device=dev))
    shape = (n_pages, n_kv, page, hd)
    for name in "kv":
        x = torch.randn(shape, generator=gen, device=dev)
        if q8:
            st[name + "_pages"], st[name + "_scales"] = _quantise(x)
        else:
            st[name + "_pages"], st[name + "_scales"] = x.half(), None
        del x
    if case["op"] == "attn":
        # fp32 queries are rows of the projections' q | k | v output, binary16 ones a buffer of their own
        wide = (n_q + 2 * n_kv) * hd if case["q"] == "f32" else n_q * hd
        q = torch.randn((rows, wide), generator=gen, device=dev) * 1.5
        st["q"], st["ld"] = (q if case["q"] == "f32" else q.half()), wide
        st["out"] = torch.zeros((rows, n_q * hd), dtype=torch.float16, device=dev)
    else:
        kv = n_kv * hd
        t = torch.float32 if case["src"] == "f32" else torch.float16
        st["ld"] = wide = (n_q + 2 * n_kv) * hd if case["src"] == "f32" and case["op"] != "read" else 2 * kv
        st["rows_kv"] = torch.zeros((rows, wide), dtype=t, device=dev) if case["op"] == "read" else torch.randn((rows, wide), generator=gen, device=dev).to(t)
        st["k_at"], st["v_at"] = wide - 2 * kv, wide - kv
        if case["op"] == "requant":
            st["back"] = torch.zeros((rows, 2 * kv), dtype=torch.float16, device=dev)
    if own:
        import weight_streaming_q4_gb300 as q4
        kind = q4.Q4_KV_Q8 if q8 else q4.Q4_KV_F16
        st["kv"] = q4.PagedKV.of(st["k_pages"], st["v_pages"], n_pages, page, n_kv, hd, kind, st["k_scales"], st["v_scales"])
        st["batch"] = q4.PagedBatch.of(st["starts"], st["lens"], st["table"], len(new), rows, width, max(new))
        if case["op"] == "attn":
            st["ws_bytes"] = q4.q4_attn_paged_workspace_bytes(n_q, n_kv, hd)
            st["ws"] = torch.empty(st["ws_bytes"], dtype=torch.uint8, device=dev)
    return st


def _places(st):
    """Of every new token row that belongs to a sequence: (row, page, slot, position, sequence)."""
    starts, lens = st["starts"].long(), st["lens"].long()
    row = torch.arange(st["rows"], device=starts.device)
    seq = torch.searchsorted(starts, row, right=True) - 1
    row = row[seq < lens.numel()]
    seq = seq[seq < lens.numel()]
    pos = lens[seq] - starts[seq + 1] + row
    return row, st["table"][seq, pos // st["page"]].long(), pos % st["page"], pos, seq


def _write_one(st, name):
    row, page, slot, _, _ = _places(st)
    at = st[name + "_at"]
    x = st["rows_kv"][row, at:at + st["n_kv"] * st["hd"]].float().unflatten(-1, (st["n_kv"], st["hd"]))
    if st["q8"]:
        code, d = _quantise(x)
        st[name + "_pages"][page, :, slot] = code
        st[name + "_scales"][page, :, slot] = d
    else:
        st[name + "_pages"][page, :, slot] = x.half()


def _read_one(st, name, out, at):
    row, page, slot, _, _ = _places(st)
    x = st[name + "_pages"][page, :, slot]
    x = _values(x, st[name + "_scales"][page, :, slot]) if st["q8"] else x
    out[row, at:at + st["n_kv"] * st["hd"]] = x.flatten(1).to(out.dtype)


def _gathered(st, name):
    """Every sequence's keys or values in order, fp32 [sequence][kv head][position][head_dim], padded to the longest."""
    pages = st["table"][:, :-(-st["longest"] // st["page"])].long().clamp(min=0)
    x = st[name + "_pages"][pages]
    x = _values(x, st[name + "_scales"][pages]) if st["q8"] else x
    return x.transpose(1, 2).flatten(2, 3)[:, :, :st["longest"]].float()


def _plain_attn(st):
    case, g = st["case"], st["n_q"] // st["n_kv"]
    row, _, _, pos, seq = _places(st)
    i = row - st["starts"].long()[seq]
    q = torch.zeros((st["lens"].numel(), st["new"], st["n_kv"], g, st["hd"]), device=row.device)
    q[seq, i] = st["q"][row, :st["n_q"] * st["hd"]].float().unflatten(-1, (st["n_kv"], g, st["hd"]))
    at = torch.full(q.shape[:2], -1, dtype=torch.long, device=row.device)
    at[seq, i] = pos
    t = torch.arange(st["longest"], device=row.device)
    sees = t <= at[..., None]
    if case["window"]:
        sees &= (t > at[..., None] - case["window"]) | (t < case["sinks"])
    s = q.permute(0, 2, 1, 3, 4).flatten(2, 3) @ _gathered(st, "k").transpose(-1, -2) / math.sqrt(st["hd"])
    s = s.unflatten(2, (st["new"], g)).masked_fill_(~sees[:, None, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = s.sum(-1, keepdim=True)
    o = s.flatten(2, 3) @ _gathered(st, "v") / torch.where(total == 0, 1.0, total).flatten(2, 3)
    o = o.unflatten(2, (st["new"], g)).permute(0, 2, 1, 3, 4)[seq, i]
    st["out"][row] = o.flatten(1).half()


def run(st):
    op, case = st["case"]["op"], st["case"]
    if own:
        import weight_streaming_q4_gb300 as q4
        if op == "attn":
            kind = q4.Q4_TYPE_F32 if case["q"] == "f32" else q4.Q4_TYPE_F16
            q4.q4_attn_paged(st["kv"], st["batch"], st["q"], kind, st["ld"], st["n_q"], case["window"], case["sinks"], st["out"], st["n_q"] * st["hd"],
                             st["ws"], st["ws_bytes"])
            return st["out"]
        kind = q4.Q4_TYPE_F32 if case["src"] == "f32" else q4.Q4_TYPE_F16
        x, ld, wide = st["rows_kv"], st["ld"], st["n_kv"] * st["hd"]
        base = x.data_ptr()
        k, v = base + st["k_at"] * x.element_size(), base + st["v_at"] * x.element_size()
        if op == "read":
            q4.q4_paged_read(st["kv"], st["batch"], k, v, kind, ld)
            return x
        q4.q4_paged_write(st["kv"], st["batch"], k, v, kind, ld)
        if op == "write":
            return {"k": st["k_pages"], "v": st["v_pages"]}
        back = st["back"].data_ptr()
        q4.q4_paged_read(st["kv"], st["batch"], back, back + 2 * wide, q4.Q4_TYPE_F16, 2 * wide)
        return st["back"]
    if op == "attn":
        _plain_attn(st)
        return st["out"]
    if op == "read":
        _read_one(st, "k", st["rows_kv"], st["k_at"])
        _read_one(st, "v", st["rows_kv"], st["v_at"])
        return st["rows_kv"]
    _write_one(st, "k")
    _write_one(st, "v")
    if op == "write":
        return {"k": st["k_pages"], "v": st["v_pages"]}
    _read_one(st, "k", st["back"], 0)
    _read_one(st, "v", st["back"], st["n_kv"] * st["hd"])
    return st["back"]


def exact(case, seed):
    if work(case)["flops"] > 8e11:
        return None
    st = prepare(case, seed)
    new, total = lengths(case)
    n_q, n_kv, hd, page = st["n_q"], st["n_kv"], st["hd"], st["page"]
    table = st["table"].cpu().tolist()

    def position_rows(name, s, length):
        """Sequence s's stored values, [kv head][position][head_dim] in 64 bits (zeros where a page was given back)."""
        parts = []
        for j in range(-(-length // page)):
            p = table[s][j]
            if p < 0:
                parts.append(torch.zeros((n_kv, page, hd), dtype=torch.float64, device="cuda"))
            elif st["q8"]:
                d = st[name + "_scales"][p].double().repeat_interleave(32, dim=-1)
                parts.append((st[name + "_pages"][p].double() * d).half().double())
            else:
                parts.append(st[name + "_pages"][p].double())
        return torch.cat(parts, dim=1)[:, :length]

    def requantised(x):
        """The value each 32-bit or 16-bit entry of x [tokens][n_kv * hd] has after Q8, from the definition in 64 bits."""
        b = x.double().reshape(x.shape[0], -1, 32)
        d = (b.abs().amax(-1, keepdim=True) / 127).half().double()
        ok = d > 0
        code = torch.where(ok, (b / torch.where(ok, d, 1.0)).round().clamp(-127, 127), 0.0)
        return (code * d).half().double().reshape(x.shape)

    if case["op"] == "attn":
        out = torch.zeros((st["rows"], n_q * hd), dtype=torch.float64, device="cuda")
        row = 0
        for s, (n, length) in enumerate(zip(new, total)):
            k, v = position_rows("k", s, length), position_rows("v", s, length)
            q = st["q"][row:row + n, :n_q * hd].double().reshape(n, n_q, hd)
            p = torch.arange(length - n, length, device="cuda")[:, None]
            t = torch.arange(length, device="cuda")[None]
            hidden = t > p
            if case["window"]:
                hidden |= (t <= p - case["window"]) & (t >= case["sinks"])
            for h in range(n_q):
                g = h // (n_q // n_kv)
                scores = (q[:, h] @ k[g].T / math.sqrt(hd)).masked_fill(hidden, -math.inf)
                out[row:row + n, h * hd:(h + 1) * hd] = torch.softmax(scores, dim=-1) @ v[g]
            row += n
        return out
    wide = n_kv * hd
    if case["op"] == "write":
        pools = {"k": st["k_pages"].double(), "v": st["v_pages"].double()}
        row = 0
        for s, (n, length) in enumerate(zip(new, total)):
            for i in range(n):
                p = length - n + i
                for name in "kv":
                    x = st["rows_kv"][row + i, st[name + "_at"]:st[name + "_at"] + wide].double()
                    pools[name][table[s][p // page], :, p % page] = x.reshape(n_kv, hd)
            row += n
        return pools
    out = torch.zeros((st["rows"], st["ld"] if case["op"] == "read" else 2 * wide), dtype=torch.float64, device="cuda")
    row = 0
    for s, (n, length) in enumerate(zip(new, total)):
        for i, name in enumerate("kv"):
            if case["op"] == "read":
                x = position_rows(name, s, length)[:, length - n:].transpose(0, 1).reshape(n, wide)
                at = st[name + "_at"]
            else:
                x, at = requantised(st["rows_kv"][row:row + n, st[name + "_at"]:st[name + "_at"] + wide]), i * wide
            out[row:row + n, at:at + wide] = x
        row += n
    return out
