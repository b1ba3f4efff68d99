"""Cases of the operators that carry a serving layer from product to product: the normalisation that prepares a sparse
product's activations, the write of new keys and values into a paged cache, attention over that cache, and attention
with a sliding window whose first tokens stay visible.

``own`` selects who computes: the plain forms below (elementary torch operations in float32; the norm's mean and the
angles in float64) or this repository's kernels. Both take the same state. Sizes are those of the layers this repository
benchmarks (Llama-3.1-8B-shaped: hidden 4096, 32 query and 8 key heads of 128; Qwen2.5-7B-shaped: hidden 3584, 28
query and 4 key heads of 128) and generic ragged ones.
"""
import math
import random

import torch

own = False
DEV = "cuda"
BF16, F32, I32, F64 = torch.bfloat16, torch.float32, torch.int32, torch.float64
FP8 = torch.float8_e4m3fn
EPS = 1e-5
BASE = 500000.0


def _pkg():
    import structured_sparse_quantized_amd as ss
    return ss


# ---- cases ---------------------------------------------------------------------------------------------------


def _norm(name, M, K, x, res, y, n):
    """x: type of the rows; y: "bf16", or "i8" / "fp8" codes lifted by the pattern (2n-2):2n (n = 2: no lift)."""
    return {"name": name, "op": "norm", "M": M, "K": K, "x": x, "res": res, "y": y, "n": n}


def _store(name, B, T, Hq, Hkv, D, rot, layout, page, start, mix):
    return {"name": name, "op": "store", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "layout": layout,
            "page": page, "start": start, "mix": mix}


def _attn(name, op, B, T, keys, longest, Hq, Hkv, D, page, window, sinks, mix):
    """B sequences with T new tokens and `keys` cached ones in all (the new ones among them), none with more than `longest`.
    op "paged": in pages of `page`; "packed": prompts without a cache; "cache": contiguous caches with room. window 0: none."""
    return {"name": name, "op": op, "B": B, "T": T, "keys": keys, "longest": longest, "Hq": Hq, "Hkv": Hkv, "D": D,
            "page": page, "window": window, "sinks": sinks, "mix": mix}


def listed():
    return [
        # one token of a decode step before the 6:8 INT8 query/key/value product: latency
        _norm("norm 1 token int8 6:8", 1, 3584, "bf16", True, "i8", 4),
        # rows of an odd size in float32 without a residual, lifted for 8:10 weights
        _norm("norm ragged f32 fp8 8:10", 777, 1501, "f32", False, "fp8", 5),
        # a long batch of prompts through the norm before the feed-forward product
        _norm("norm 16384 tokens fp8", 16384, 4096, "bf16", True, "fp8", 2),
        # the next token of a small serving batch into its pages: latency
        _store("store 4 tokens", 4, 4, 32, 8, 128, 128, "half", 16, 4000, 1),
        # queries, keys and values of a packed batch of prompts, some with cached text before them
        _store("store 8192 tokens", 9, 8192, 28, 4, 128, 128, "half", 64, 1500, 2),
        # the next token of one sequence over its pages: latency
        _attn("paged 1 token", "paged", 1, 1, 4000, 4096, 32, 8, 128, 16, 0, 0, 3),
        # the next tokens of a serving batch, caches filled to very different lengths
        _attn("paged 64 caches", "paged", 64, 64, 262144, 8192, 32, 8, 128, 16, 0, 0, 4),
        # a few drafted tokens of each sequence at once, heads of 80, pages of an odd size
        _attn("paged drafts ragged", "paged", 13, 61, 30011, 6000, 12, 4, 80, 24, 0, 0, 5),
        # long conversations of which a window and the first tokens stay: the pages between them are given back
        _attn("paged window 32 caches", "paged", 32, 32, 800000, 32768, 28, 4, 128, 32, 4096, 4, 6),
        # a serving batch over contiguous caches, the last 1000 keys of each
        _attn("window 24 caches", "cache", 24, 24, 100000, 8192, 32, 8, 128, 0, 1000, 0, 7),
        # a packed batch of prompts of different lengths, heads of 64, a short window
        _attn("window packed prompts", "packed", 9, 8001, 8001, 4000, 12, 12, 64, 0, 300, 0, 8),
        # one long prompt, a window and four first tokens
        _attn("window 8192 prompt", "packed", 1, 8192, 8192, 8192, 32, 8, 128, 0, 1024, 4, 9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "store", "paged", "paged", "cache", "packed"))
    mix = rng.randrange(1 << 20)
    if op == "norm":
        K = _log(rng, 64, 18944)
        y = rng.choice(("bf16", "i8", "fp8"))
        c = _norm("", max(1, _log(rng, 1, max(2, 16384 * 2048 // K))), K, rng.choice(("bf16", "bf16", "f32")), rng.random() < 0.6, y,
                  2 if y == "bf16" else rng.choice((2, 2, 3, 4, 5)))
        c["M"] = min(c["M"], 16384)
    elif op == "store":
        D = rng.choice((32, 64, 80, 96, 128))
        Hkv = rng.choice((1, 2, 4, 8))
        Hq = Hkv * rng.choice((1, 2, 4, 7))
        B = _log(rng, 1, 64)
        c = _store("", B, B if rng.random() < 0.5 else _log(rng, B, max(B + 1, 6000)), Hq, Hkv, D,
                   D if rng.random() < 0.5 else 2 * rng.randint(1, D // 2), rng.choice(("half", "interleaved")),
                   rng.choice((1, 16, 24, 32, 64, 128)), rng.choice((0, _log(rng, 1, 4000))), mix)
    else:
        D = rng.choice((32, 64, 80, 96, 128, 128))
        Hkv = rng.choice((1, 2, 4, 8))
        Hq = Hkv * rng.choice((1, 2, 4, 5, 7, 8))
        if Hq * D > 4096:
            Hq = max(Hkv, 4096 // D // Hkv * Hkv)
        window = _log(rng, 1, 4096) if op != "paged" or rng.random() < 0.5 else 0
        sinks = rng.choice((0, 1, 4, 16, 100)) if window else 0
        if op == "packed":
            B = _log(rng, 1, 32)
            T = max(B, _log(rng, 16, 8000))
            c = _attn("", op, B, T, T, T, Hq, Hkv, D, 0, window, sinks, mix)
        else:
            B = _log(rng, 1, 64)
            longest = _log(rng, 16, 8192)
            keys = B * min(_log(rng, 1, longest), 262144 // B)
            c = _attn("", op, B, B if rng.random() < 0.7 else B * rng.randint(2, 9), keys, longest, Hq, Hkv, D,
                      rng.choice((1, 16, 24, 32, 64, 128)) if op == "paged" else 0, window, sinks, mix)
    del c["name"]
    return c


def _share(r, total, parts):
    """`total` in `parts` uneven shares of at least one."""
    w = [r.uniform(0.2, 1.0) for _ in range(parts)]
    n = [max(1, int(total * x / sum(w))) for x in w]
    n[-1] = max(1, total - sum(n[:-1]))
    return n


def _lens(c):
    """New tokens and keys (the new ones among them) of each sequence. A sequence of a cache may hold less than its new
    tokens: the first of them then see nothing."""
    r = random.Random(c["mix"])
    B = c["B"]
    lq = [1] * B if c["T"] == B else _share(r, c["T"], B)
    if c["op"] == "packed":
        return lq, list(lq)
    if c["op"] == "store":
        return lq, [n + (r.randint(0, 2 * c["start"]) if B > 1 else c["start"]) for n in lq]
    if B == 1:
        return lq, [min(c["keys"], c["longest"])]
    mean = c["keys"] / B
    spread = min(mean - 1, c["longest"] - mean)
    return lq, [int(round(mean + spread * r.uniform(-1, 1))) for _ in range(B)]


def _seen(c):
    """(pairs of a new token and a key that it sees, keys that some new token sees), all sequences."""
    pairs = keys = 0
    w, s = c["window"] or 1 << 40, c["sinks"]
    for a, b in zip(*_lens(c)):
        for p in range(max(b - a, 0), b):
            pairs += min(p + 1, w) + min(max(p + 1 - w, 0), s)
        low = max(max(b - a, 0) - w + 1, 0)  # of the first row that sees anything
        keys += b - low + min(low, s)
    return pairs, keys


def work(c):
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        es = 4 if c["x"] == "f32" else 2
        out = 2 * K if c["y"] == "bf16" else _lifted(K, c["n"]) + 4
        return {"bytes": M * (K * es * (3 if c["res"] else 1) + out) + 4 * K, "flops": 6 * M * K}
    if c["op"] == "store":
        n = c["T"] * (c["Hq"] + 2 * c["Hkv"])
        return {"bytes": 4 * n * c["D"] + 8 * c["T"], "flops": 3 * c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"]}
    pairs, keys = _seen(c)
    D = c["D"]
    return {"bytes": 4 * D * (c["T"] * c["Hq"] + keys * c["Hkv"]), "flops": 4 * D * c["Hq"] * pairs}


# ---- states --------------------------------------------------------------------------------------------------


def _lifted(K, n):
    return ((K + 2 * n - 1) // (2 * n) * 4 * (n - 1) + 255) // 256 * 256


def _ints(v):
    return torch.tensor(v, dtype=I32).to(DEV)


def _cumulative(n):
    return [sum(n[:i]) for i in range(len(n) + 1)]


def _prepare_norm(c, g):
    M, K = c["M"], c["K"]
    t = F32 if c["x"] == "f32" else BF16
    ld = (K + 7) // 8 * 8  # rows start on 16 bytes
    # channels of very different sizes, as residual streams have them
    size = torch.exp(torch.randn(K, generator=g, device=DEV))
    rows = lambda: torch.randn((M, ld), generator=g, device=DEV)[:, :K]  # noqa: E731
    st = {"res": (rows() * size).to(t) if c["res"] else None}
    x = rows() * (1.0 if c["res"] else size)
    st["x"] = torch.zeros((M, ld), dtype=t, device=DEV)[:, :K].copy_(x)
    if c["res"]:
        st["res"] = torch.zeros((M, ld), dtype=t, device=DEV)[:, :K].copy_(st["res"])
    st["w"] = (1 / size * (0.5 + torch.rand(K, generator=g, device=DEV))).to(t)
    return st


def _frequencies(rot):
    """Radians a position turns each pair."""
    return BASE ** (-2 * torch.arange(rot // 2, dtype=F64) / rot)


def _table(r, c, need, spare):
    """Pages for `need[b]` keys of each sequence, in an order of the pool's own; unused entries name no page."""
    used = [(n + c["page"] - 1) // c["page"] for n in need]
    free = list(range(sum(used) + spare))
    r.shuffle(free)
    wide = max(max(used), 1) + 2
    return [[free.pop() for _ in range(n)] + [-1] * (wide - n) for n in used], sum(used) + spare


def _prepare_store(c, g):
    lq, lk = _lens(c)
    T, Hq, Hkv, D, page = sum(lq), c["Hq"], c["Hkv"], c["D"], c["page"]
    table, pages = _table(random.Random(c["mix"] + 1), c, lk, 3)
    row = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=DEV).to(BF16).unflatten(1, (Hq + 2 * Hkv, D))
    f = _frequencies(c["rot"])
    turns = [int(x / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for x in f.tolist()]  # 2^-64 turns a position
    pool = torch.randn((2, pages, page, Hkv, D), generator=g, device=DEV).to(BF16)
    return {"q": row[:, :Hq], "k": row[:, Hq : Hq + Hkv], "v": row[:, Hq + Hkv :], "freq": f.to(DEV),
            "steps": torch.tensor([x - (1 << 64) if x >> 63 else x for x in turns], dtype=torch.int64).to(DEV),
            "pos": _ints([b - a + i for a, b in zip(lq, lk) for i in range(a)]), "layout": c["layout"],
            "cu": None if T == c["B"] else _ints(_cumulative(lq)), "table": _ints(table), "kp": pool[0], "vp": pool[1]}


def _prepare_attn(c, g):
    lq, lk = _lens(c)
    B, Hq, Hkv, D, w, s = c["B"], c["Hq"], c["Hkv"], c["D"], c["window"], c["sinks"]
    T = sum(lq)
    st = {"cu_q": _ints(_cumulative(lq)), "max_q": max(lq), "max_k": max(lk), "window": w, "sinks": s}
    if c["op"] == "packed":  # heads of one projection's output, side by side
        row = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=DEV).to(BF16).unflatten(1, (Hq + 2 * Hkv, D))
        st["q"], st["k"], st["v"] = row[:, :Hq], row[:, Hq : Hq + Hkv], row[:, Hq + Hkv :]
        st["cu_k"], st["k_len"] = st["cu_q"], None
        return st
    st["q"] = torch.randn((T, Hq, D), generator=g, device=DEV).to(BF16)
    st["k_len"] = _ints(lk)
    if c["op"] == "cache":
        room = c["longest"]
        st["k"], st["v"] = (torch.randn((B * room, Hkv, D), generator=g, device=DEV).to(BF16) for _ in range(2))
        st["cu_k"] = _ints([b * room for b in range(B + 1)])
        return st
    page = c["page"]
    table, pages = _table(random.Random(c["mix"] + 1), c, lk, 2)
    if w:  # pages that no new token sees any more are given back
        for row, a, b in zip(table, lq, lk):
            for i in range((s + page - 1) // page, max(max(b - a, 0) - w + 1, 0) // page):
                row[i] = -1
    st["table"] = _ints(table)
    st["kp"], st["vp"] = (torch.randn((pages, page, Hkv, D), generator=g, device=DEV).to(BF16) for _ in range(2))
    return st


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"norm": _prepare_norm, "store": _prepare_store}.get(c["op"], _prepare_attn)(c, g)
    st["case"] = c
    return st


# ---- one pass ------------------------------------------------------------------------------------------------


def _plain_norm(st):
    c, x = st["case"], st["x"].float()
    r = st["x"] if st["res"] is None else (x + st["res"].float()).to(st["x"].dtype)
    rs = (1 / torch.sqrt(r.double().square().mean(1, keepdim=True) + EPS)).float()
    z = r.float() * rs * st["w"].float()
    out = {} if st["res"] is None else {"sum": r}
    if c["y"] == "bf16":
        return {"y": z.to(BF16), **out}
    top = 127.0 if c["y"] == "i8" else 448.0
    a = z.abs().amax(1, keepdim=True)
    t = (z * torch.where(a > 0, top / a, 0.0)).clamp_(-top, top)
    q = (t.round_().to(torch.int8) if c["y"] == "i8" else t.to(FP8)).view(torch.int8)
    # the lift: window w of group g takes the group's positions 2w .. 2w + 3
    n, K, Kc = c["n"], c["K"], _lifted(c["K"], c["n"])
    at = torch.arange(Kc, device=DEV)
    src = at // (4 * (n - 1)) * (2 * n) + at % (4 * (n - 1)) // 4 * 2 + at % 4
    y = torch.where(src < K, q[:, src.clamp(max=K - 1)], 0)
    # the codes: whole numbers, or floats of 8 bits; times their row's scale they are the values
    return {"y": y.view(torch.int8 if c["y"] == "i8" else FP8), "scale": (a / top).squeeze(1), **out}


def _turned(x, pos, freq, layout):
    rot = 2 * freq.numel()
    angle = pos.double()[:, None, None] * freq
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    x = x.float()
    a, b = (x[..., : rot // 2], x[..., rot // 2 : rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat((u, v), -1) if layout == "half" else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1).to(BF16)


def _plain_store(st):
    pos, page = st["pos"].long(), st["case"]["page"]
    T = pos.numel()
    tok = torch.arange(T, device=DEV)
    seq = tok if st["cu"] is None else (tok[:, None] >= st["cu"][1:]).sum(1)
    entry = st["table"][seq, pos // page].long()
    st["kp"][entry, pos % page] = _turned(st["k"], st["pos"], st["freq"], st["layout"])
    st["vp"][entry, pos % page] = st["v"]
    return {"q": _turned(st["q"], st["pos"], st["freq"], st["layout"]), "k": st["kp"], "v": st["vp"]}


def _plain_attn(st):
    c, q, cu_q = st["case"], st["q"], st["cu_q"].long()
    T, Hq, D = q.shape
    Hkv, B, mq, mk = c["Hkv"], c["B"], st["max_q"], max(st["max_k"], 1)
    lq = cu_q[1:] - cu_q[:-1]
    iq, ik = torch.arange(mq, device=DEV), torch.arange(mk, device=DEV)
    rq = (cu_q[:-1, None] + iq).clamp(max=T - 1)  # padded: [B, mq] rows, [B, mk] keys
    if c["op"] == "paged":
        lk = st["k_len"].long()
        entry = st["table"][:, ik // c["page"]].long()
        there = entry >= 0
        k, v = (t[entry.clamp(min=0), ik % c["page"]] for t in (st["kp"], st["vp"]))
    else:
        cu_k = st["cu_k"].long()
        lk = st["k_len"].long() if st["k_len"] is not None else cu_k[1:] - cu_k[:-1]
        rk = (cu_k[:-1, None] + ik).clamp(max=st["k"].shape[0] - 1)
        there = torch.ones((1, 1), dtype=torch.bool, device=DEV)
        k, v = st["k"][rk], st["v"][rk]
    qp = q[rq].float().unflatten(2, (Hkv, Hq // Hkv)).permute(0, 2, 3, 1, 4).reshape(B * Hkv, -1, D)
    kp, vp = (t.float().transpose(1, 2).reshape(B * Hkv, mk, D) for t in (k, v))
    s = torch.bmm(qp, kp.transpose(1, 2).contiguous()).mul_(1 / math.sqrt(D)).view(B, Hkv, -1, mq, mk)
    at = (iq + (lk - lq)[:, None])[..., None]  # the row's position
    seen = (ik <= at) & (ik < lk[:, None, None]) & there[:, None]
    if st["window"]:
        seen = seen & ((ik > at - st["window"]) | (ik < st["sinks"]))
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    n = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(B * Hkv, -1, mk), vp).view(B, Hkv, -1, mq, D) / torch.where(n > 0, n, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, mq, Hq, D)
    return o[iq < lq[:, None]].to(q.dtype)


def _own_norm(st):
    c = st["case"]
    y, scale, total = _pkg().rmsnorm_act(st["x"], st["w"], EPS, residual=st["res"], n=c["n"], y_dtype=c["y"])
    out = {} if total is None else {"sum": total}
    return {"y": y, **out} if scale is None else {"y": y, "scale": scale, **out}


def _own_store(st):
    q = _pkg().paged_store(st["k"], st["v"], st["pos"], st["kp"], st["vp"], st["table"], cu=st["cu"], q=st["q"], steps=st["steps"],
                           layout=st["layout"])
    return {"q": q, "k": st["kp"], "v": st["vp"]}


def _own_attn(st):
    ss, window = _pkg(), st["window"] or None
    if st["case"]["op"] == "paged":
        return ss.attn_paged(st["q"], st["kp"], st["vp"], st["table"], st["k_len"], cu_q=st["cu_q"], window=window,
                             sinks=st["sinks"])
    return ss.attn(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], k_len=st["k_len"], window=window, sinks=st["sinks"])


def run(st):
    op = st["case"]["op"]
    if own:
        return {"norm": _own_norm, "store": _own_store}.get(op, _own_attn)(st)
    return {"norm": _plain_norm, "store": _plain_store}.get(op, _plain_attn)(st)


# ---- the definitions in 64 bits ----------------------------------------------------------------------------


def _exact_norm(c, st):
    r = st["x"].double()
    out = {}
    if st["res"] is not None:
        out["sum"] = r + st["res"].double()
        r = out["sum"].to(st["x"].dtype).double()  # the stream as it is kept
    power = torch.linalg.vector_norm(r, dim=1, keepdim=True) ** 2 / c["K"]
    z = st["w"].double() * r * (power + EPS) ** -0.5
    if c["y"] == "bf16":
        return {"y": z, **out}
    top = 127 if c["y"] == "i8" else 448
    scale = torch.linalg.vector_norm(z, ord=math.inf, dim=1) / top
    out["scale"] = scale
    if c["y"] == "fp8":
        n, groups = c["n"], -(-c["K"] // (2 * c["n"]))
        codes = (z / scale[:, None]).to(F32).to(FP8).double()
        padded = torch.nn.functional.pad(codes, (0, groups * 2 * n - c["K"])).view(c["M"], groups, 2 * n)
        lifted = padded.unfold(2, 4, 2).reshape(c["M"], -1)  # overlapping windows of four, two apart
        out["y"] = torch.nn.functional.pad(lifted, (0, _lifted(c["K"], n) - lifted.shape[1]))
    else:
        out["y"] = None  # whole numbers
    return out


def _exact_store(c, st):
    lq, lk = _lens(c)
    n = c["rot"] // 2
    re, im = (slice(0, n), slice(n, 2 * n)) if c["layout"] == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))

    def turn(x):
        out = x.double().clone()
        z = torch.complex(out[..., re], out[..., im])
        z = z * torch.polar(torch.ones((), dtype=F64, device=DEV), torch.outer(st["pos"].double(), st["freq"]))[:, None]
        out[..., re], out[..., im] = z.real, z.imag
        return out

    q, k, v = turn(st["q"]), turn(st["k"]), st["v"].double()
    kp, vp = st["kp"].double(), st["vp"].double()
    table = st["table"].tolist()
    place = []
    for row, a, b in zip(table, lq, lk):
        place += [row[p // c["page"]] * c["page"] + p % c["page"] for p in range(b - a, b)]
    place = torch.tensor(place, device=DEV)
    for pool, rows in ((kp, k), (vp, v)):
        pool.view(-1, c["Hkv"], c["D"]).index_copy_(0, place, rows)
    return {"q": q, "k": kp, "v": vp}


def _exact_attn(c, st):
    lq, lk = _lens(c)
    G, D = c["Hq"] // c["Hkv"], c["D"]
    out = torch.zeros(st["q"].shape, dtype=F64, device=DEV)
    at = 0
    for i, (a, b) in enumerate(zip(lq, lk)):
        first = max(0, a - b)  # rows before it see nothing
        for r0 in range(first, a, 1024):
            r1 = min(a, r0 + 1024)
            lo, hi = r0 + b - a, r1 + b - a  # positions of these rows
            low = max(0, lo - c["window"] + 1) if c["window"] else 0
            idx = torch.cat((torch.arange(min(c["sinks"], low), device=DEV), torch.arange(low, hi, device=DEV)))
            if c["op"] == "paged":
                rows = st["table"][i].long()[idx // c["page"]] * c["page"] + idx % c["page"]
                k, v = (t.view(-1, c["Hkv"], D)[rows].double() for t in (st["kp"], st["vp"]))
            else:
                k, v = (t[int(st["cu_k"][i]) + idx].double() for t in (st["k"], st["v"]))
            pos = torch.arange(lo, hi, device=DEV)[:, None]
            hidden = idx > pos
            if c["window"]:
                hidden = hidden | ((pos - idx >= c["window"]) & (idx >= c["sinks"]))
            for h in range(c["Hkv"]):
                x = st["q"][at + r0 : at + r1, h * G : (h + 1) * G].double().transpose(0, 1)
                score = (x @ k[:, h].t().contiguous()) / math.sqrt(D)
                w = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
                out[at + r0 : at + r1, h * G : (h + 1) * G] = (w @ v[:, h]).transpose(0, 1)
        at += a
    return out


def exact(c, seed):
    st = prepare(c, seed)
    return {"norm": _exact_norm, "store": _exact_store}.get(c["op"], _exact_attn)(c, st)
