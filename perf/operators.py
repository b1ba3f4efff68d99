"""Cases of the operators around the sparse products of a transformer layer: the product with its epilogue
(bias, activation, gate, residual), rotary positions, and attention over packed sequences and caches.

``own`` selects who computes: the plain forms below (elementary torch operations in float32, angles in float64)
or this repository's kernels. Both take the same state. Sizes are those of the layers this repository
benchmarks (Llama-3.1-8B-shaped: hidden 4096, 32 query and 8 key heads of 128, feed-forward 14336;
Qwen2.5-7B-shaped: hidden 3584, 28 query and 4 key heads of 128) and generic ragged ones.
"""
import math
import random

import torch

own = False
DEV = "cuda"
PAIRS = ((0, 1), (0, 2), (0, 3), (1, 2), (1, 3), (2, 3))  # the six ways to keep two of four positions
BF16, F32 = torch.bfloat16, torch.float32


def _pkg():
    import structured_sparse_quantized_amd as ss
    return ss


# ---- cases ---------------------------------------------------------------------------------------------------


def _product(name, side, ab, M, N, K, bias=False, act="none", gated=False, res=False, y="bf16"):
    return {"name": name, "op": "product", "side": side, "ab": ab, "M": M, "N": N, "K": K, "bias": bias, "act": act,
            "gated": gated, "res": res, "y": y}


def _rotary(name, T, H, D, rot, layout, x, scaling, start):
    return {"name": name, "op": "rotary", "T": T, "H": H, "D": D, "rot": rot, "layout": layout, "x": x,
            "scaling": scaling, "start": start}


def _attn(name, kind, B, total, cap, Hq, Hkv, D, causal, mix):
    return {"name": name, "op": "attn", "kind": kind, "B": B, "total": total, "cap": cap, "Hq": Hq, "Hkv": Hkv, "D": D,
            "causal": causal, "mix": mix}


def listed():
    return [
        # one token through the query/key/value projection, whose channels carry biases: latency
        _product("bias 1 token int8", "W", "i8", 1, 4608, 3584, bias=True, y="f32"),
        # a serving batch through the attention output projection, added to the residual stream
        _product("residual 48 tokens fp8", "W", "fp8", 48, 4096, 4096, res=True),
        # a prompt through the gate and up projection, gated in the epilogue: half the outputs leave
        _product("gate 4096 tokens fp8", "W", "fp8", 4096, 28672, 4096, act="silu", gated=True),
        # pruned activations times dense bf16 weights of an odd size, bias, GELU and residual
        _product("gelu sparse x ragged bf16", "X", "bf16", 777, 1001, 1500, bias=True, act="gelu_tanh", res=True),
        # the next position of one sequence: queries and keys of one token, context scaled for length: latency
        _rotary("rotary 1 token", 1, 40, 128, 128, "half", "bf16", "smooth", 90000),
        # part of each head, interleaved pairs, float32, an odd count of tokens far into a context
        _rotary("rotary part of the head f32", 777, 14, 80, 32, "interleaved", "f32", "none", 1000000),
        # the queries and keys of a long prompt
        _rotary("rotary 16384 tokens", 16384, 40, 128, 128, "half", "bf16", "yarn", 0),
        # the next token of one sequence over its cache: latency
        _attn("attention 1 token", "decode", 1, 4000, 4096, 32, 8, 128, True, 1),
        # the next tokens of a serving batch, caches filled to different lengths
        _attn("attention 64 caches", "decode", 64, 262144, 8192, 32, 8, 128, True, 2),
        # a packed batch of prompts of different lengths, seven query heads to a key head
        _attn("attention packed prompts", "prompt", 9, 8001, 0, 28, 4, 128, True, 3),
        # queries over the keys of another text, heads of 64, some of them without any key
        _attn("attention cross ragged", "cross", 13, 2500, 1777, 12, 12, 64, False, 4),
        # one long prompt
        _attn("attention 8192 prompt", "prompt", 1, 8192, 0, 32, 8, 128, True, 5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("product", "rotary", "attn"))
    if op == "product":
        side = rng.choice(("W", "W", "X"))
        ab = rng.choice(("i8", "fp8", "bf16"))
        M, K = _log(rng, 1, 4096), _log(rng, 200, 14336)
        N = _log(rng, 64, min(28672, 4096 * 28672 * 4096 // (M * K)))
        gated = rng.random() < 0.3
        N += N % 2 if gated else 0
        c = _product("", side, ab, M, N, K, rng.random() < 0.6, rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")),
                     gated, rng.random() < 0.5, rng.choice(("bf16", "f32")) if ab == "i8" else "bf16")
    elif op == "rotary":
        D = rng.choice((32, 64, 80, 96, 128, 256))
        H = rng.randint(1, 5120 // D)
        rot = D if rng.random() < 0.5 else 2 * rng.randint(1, D // 2)
        x = rng.choice(("bf16", "bf16", "f32"))
        c = _rotary("", _log(rng, 1, 8192), H, D, rot, rng.choice(("half", "interleaved")), x,
                    rng.choice(("none", "linear", "ntk", "smooth", "yarn")), rng.choice((0, _log(rng, 1, 2000000))))
    else:
        kind = rng.choice(("decode", "prompt", "cross"))
        D = rng.choice((32, 64, 80, 96, 128, 128))
        Hkv = rng.choice((1, 2, 4, 8))
        Hq = Hkv * rng.choice((1, 2, 4, 5, 7, 8))
        if Hq * D > 4096:
            Hq = max(Hkv, 4096 // D // Hkv * Hkv)
        B = _log(rng, 1, 32)
        if kind == "decode":
            cap = _log(rng, 16, 8192)
            c = _attn("", kind, B, B * max(1, _log(rng, 1, cap)), cap, Hq, Hkv, D, True, rng.randrange(1 << 20))
        elif kind == "prompt":
            c = _attn("", kind, B, max(B, _log(rng, 16, 8000)), 0, Hq, Hkv, D, rng.random() < 0.8, rng.randrange(1 << 20))
        else:
            c = _attn("", kind, B, max(B, _log(rng, 16, 3000)), _log(rng, 1, 2000), Hq, Hkv, D, rng.random() < 0.4,
                      rng.randrange(1 << 20))
    del c["name"]
    return c


def _split(r, total, parts):
    """`total` in `parts` uneven shares of at least one."""
    w = [r.uniform(0.2, 1.0) for _ in range(parts)]
    n = [max(1, int(total * x / sum(w))) for x in w]
    n[-1] = max(1, total - sum(n[:-1]))
    return n


def _lens(c):
    """Query lengths, key lengths and the first key row of each sequence."""
    r = random.Random(c["mix"])
    B, total, cap = c["B"], c["total"], c["cap"]
    if c["kind"] == "prompt":
        lq = _split(r, total, B)
        return lq, lq, [sum(lq[:b]) for b in range(B)]
    if c["kind"] == "decode":
        mean = total / B
        spread = min(mean - 1, cap - mean)
        lk = [int(round(mean + spread * r.uniform(-1, 1))) for _ in range(B)]
        if B == 1:
            lk = [min(total, cap)]
        return [1] * B, [min(max(n, 1), cap) for n in lk], [b * cap for b in range(B)]
    lq = _split(r, total, B)
    lk = [0 if r.random() < 0.15 else r.randint(1, cap) for _ in range(B)]
    if not any(lk):
        lk[0] = cap
    return lq, lk, [sum(lk[:b]) for b in range(B)]


def _visible(lq, lk, causal):
    """Key rows that each query row sees, summed: with a causal mask the last query row sees the last key."""
    if not causal:
        return sum(a * b for a, b in zip(lq, lk))
    n = 0
    for a, b in zip(lq, lk):
        first = max(0, a - b)  # rows before it see nothing
        rows = a - first
        n += rows * (b - a + first + 1) + rows * (rows - 1) // 2
    return n


def work(c):
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        es = 2 if c["ab"] == "bf16" else 1
        Kc, No, yb = _pad(K), N // 2 if c["gated"] else N, 4 if c["y"] == "f32" else 2
        sparse, dense = (N, M) if c["side"] == "W" else (M, N)
        b = sparse * Kc * (es / 2 + 1 / 8) + dense * Kc * es + M * No * yb * (2 if c["res"] else 1)
        b += 4 * (M + N) * (c["ab"] != "bf16") + 4 * N * c["bias"]
        return {"bytes": b, "flops": M * N * K}  # half of the positions are kept
    if c["op"] == "rotary":
        n = c["T"] * c["H"]
        return {"bytes": 2 * n * c["D"] * (4 if c["x"] == "f32" else 2) + 4 * c["T"], "flops": 3 * n * c["rot"]}
    lq, lk, _ = _lens(c)
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    return {"bytes": 2 * D * (2 * sum(lq) * Hq + 2 * sum(lk) * Hkv), "flops": 4 * D * Hq * _visible(lq, lk, c["causal"])}


# ---- states --------------------------------------------------------------------------------------------------


def _pad(K):
    return (K + 255) // 256 * 256


def _codes(g, shape, ab):
    """Operand codes as the quantisers of this library leave them, and the size of one unit."""
    x = torch.randn(shape, generator=g, device=DEV)
    if ab == "i8":
        return (x * 32).round_().clamp_(-127, 127).to(torch.int8), 1 / 32
    if ab == "fp8":
        return (x * 112).clamp_(-448, 448).to(torch.float8_e4m3fn), 1 / 112
    return x.to(BF16), 1.0


def _sparse_codes(g, rows, K, ab):
    """A 2:4 operand [rows][Kc]: dense codes with the dropped positions zero, and values and positions as compressed."""
    Kc, KG = _pad(K), (K + 3) // 4
    vals, unit = _codes(g, (rows, Kc // 4, 2), ab)
    bits = vals.view(torch.int16 if ab == "bf16" else torch.int8)
    bits[:, KG:] = 0
    nib = torch.tensor([a | b << 2 for a, b in PAIRS], dtype=torch.uint8, device=DEV)
    kind = torch.randint(0, 6, (rows, Kc // 4), generator=g, device=DEV)
    kind[:, KG:] = 0
    pos = torch.tensor(PAIRS, device=DEV)[kind]
    dense = torch.zeros((rows, Kc // 4, 4), dtype=bits.dtype, device=DEV).scatter_(2, pos, bits)
    half = nib[kind].view(rows, Kc // 8, 2)
    meta = (half[..., 0] | half[..., 1] << 4).contiguous()
    return dense.view(rows, Kc).view(vals.dtype), bits.view(rows, Kc // 2).view(vals.dtype), meta, unit


def _prepare_product(c, g):
    M, N, K, ab = c["M"], c["N"], c["K"], c["ab"]
    sparse, dense = (N, M) if c["side"] == "W" else (M, N)
    sp, vals, meta, unit = _sparse_codes(g, sparse, K, ab)
    dn, _ = _codes(g, (dense, _pad(K)), ab)
    dn.view(torch.int16 if ab == "bf16" else torch.int8)[:, K:] = 0
    st = {"w": sp if c["side"] == "W" else dn, "x": dn if c["side"] == "W" else sp, "dense": dn}
    one = 1 / math.sqrt(K / 2)
    if ab == "bf16":
        st["sx"] = st["sw"] = None
        if c["side"] == "W":  # weights of the size that keeps the outputs near one
            st["sw"] = torch.full((N,), one, device=DEV)
        else:
            st["w"] = st["dense"] = (dn * one).to(BF16)
    else:
        st["sx"] = unit * (0.5 + torch.rand(M, generator=g, device=DEV))
        st["sw"] = unit * one * (0.5 + torch.rand(N, generator=g, device=DEV))
    out = (M, N // 2 if c["gated"] else N)
    st["y"] = F32 if c["y"] == "f32" else BF16
    st["bias"] = 0.5 * torch.randn(N, generator=g, device=DEV) if c["bias"] else None
    st["res"] = torch.randn(out, generator=g, device=DEV).to(st["y"]) if c["res"] else None
    if own:  # the tiled operand: weights are laid out once; pruned activations arrive in this layout
        st["tv"], st["tm"] = _pkg().pack_sparse(vals, meta)
    return st


SCALING = {  # name -> (factor, original context, low, high) of the position plan
    "none": (1.0, 0, 1.0, 1.0),
    "linear": (4.0, 0, 1.0, 1.0),
    "ntk": (4.0, 0, 1.0, 1.0),
    "smooth": (8.0, 8192, 1.0, 4.0),
    "yarn": (4.0, 32768, 1.0, 32.0),
}
BASE = 500000.0


def _frequencies(rot, scaling):
    """Radians a position turns each pair, float64, and the factor on the rotated values."""
    factor, orig, low, high = SCALING[scaling]
    i = torch.arange(rot // 2, dtype=torch.float64)
    base = BASE * factor ** (rot / (rot - 2)) if scaling == "ntk" and rot > 2 else BASE
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "smooth":  # turns over the original context: few -> stretched, many -> kept
        turns = orig * f / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        f = f / factor * (1 - keep) + f * keep
    if scaling == "yarn":  # a ramp over the pairs between those that turn `high` and `low` times
        at = [rot * math.log(orig / (2 * math.pi * n)) / (2 * math.log(BASE)) for n in (high, low)]
        a, b = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
        ramp = ((i - a) / max(b - a, 0.001)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
    return f, 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0


def _prepare_rotary(c, g):
    T, H, D = c["T"], c["H"], c["D"]
    # the queries and keys of a token stand together in the projection's output, before its values
    row = torch.randn((T, (H + 8) * D), generator=g, device=DEV).to(F32 if c["x"] == "f32" else BF16)
    f, m = _frequencies(c["rot"], c["scaling"])
    st = {"x": row[:, : H * D].unflatten(1, (H, D)), "freq": f.to(DEV), "mscale": m, "layout": c["layout"]}
    st["pos"] = c["start"] + torch.randperm(T, generator=g, device=DEV).to(torch.int32)
    if own:
        factor, orig, low, high = SCALING[c["scaling"]]
        st["steps"], st["mscale"] = _pkg().rotary_steps(c["rot"], base=BASE, scaling=c["scaling"], factor=factor,
                                                        original=orig, low=low, high=high, device=DEV)
    return st


def _ints(v):
    return torch.tensor(v, dtype=torch.int32).to(DEV)


def _cumulative(n):
    return [sum(n[:i]) for i in range(len(n) + 1)]


def _prepare_attn(c, g):
    lq, lk, start = _lens(c)
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    st = {"cu_q": _ints(_cumulative(lq)), "max_q": max(lq), "max_k": max(lk), "causal": c["causal"], "k_len": None}
    if c["kind"] == "prompt":  # heads of one projection's output, side by side
        T = sum(lq)
        row = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=DEV).to(BF16).unflatten(1, (Hq + 2 * Hkv, D))
        st["q"], st["k"], st["v"] = row[:, :Hq], row[:, Hq : Hq + Hkv], row[:, Hq + Hkv :]
        st["cu_k"] = st["cu_q"]
        return st
    Tk = B * c["cap"] if c["kind"] == "decode" else sum(lk)
    st["q"] = torch.randn((sum(lq), Hq, D), generator=g, device=DEV).to(BF16)
    st["k"], st["v"] = (torch.randn((Tk, Hkv, D), generator=g, device=DEV).to(BF16) for _ in range(2))
    st["cu_k"] = _ints(start + [Tk])
    if c["kind"] == "decode":
        st["k_len"] = _ints(lk)
    return st


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"product": _prepare_product, "rotary": _prepare_rotary, "attn": _prepare_attn}[c["op"]](c, g)
    st["case"] = c
    return st


# ---- one pass ------------------------------------------------------------------------------------------------


def _act(v, name):
    if name == "relu":
        return v.clamp_min(0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_product(st):
    c = st["case"]
    y = st["x"].float() @ st["w"].float().t()
    if st["sx"] is not None:
        y = y * st["sx"][:, None]
    if st["sw"] is not None:
        y = y * st["sw"]
    if st["bias"] is not None:
        y = y + st["bias"]
    y = _act(y[:, 0::2], c["act"]) * y[:, 1::2] if c["gated"] else _act(y, c["act"])
    if st["res"] is not None:
        y = y + st["res"].float()
    return y.to(st["y"])


def _plain_rotary(st):
    x, rot = st["x"].float(), 2 * st["freq"].numel()
    angle = st["pos"].double()[:, None, None] * st["freq"]
    cos, sin = ((f(angle) * st["mscale"]).float() for f in (torch.cos, torch.sin))
    a, b = (x[..., : rot // 2], x[..., rot // 2 : rot]) if st["layout"] == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat((u, v), -1) if st["layout"] == "half" else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1).to(st["x"].dtype)


def _plain_attn(st):
    q, k, v, cu_q, cu_k = st["q"], st["k"], st["v"], st["cu_q"].long(), st["cu_k"].long()
    T, Hq, D = q.shape
    Hkv, B, mq, mk = k.shape[1], cu_q.numel() - 1, st["max_q"], st["max_k"]
    lq = cu_q[1:] - cu_q[:-1]
    lk = st["k_len"].long() if st["k_len"] is not None else cu_k[1:] - cu_k[:-1]
    iq, ik = torch.arange(mq, device=DEV), torch.arange(mk, device=DEV)
    rq = (cu_q[:-1, None] + iq).clamp(max=T - 1)  # padded: [B, mq] rows, [B, mk] keys
    rk = (cu_k[:-1, None] + ik).clamp(max=k.shape[0] - 1)
    qp = q[rq].float().unflatten(2, (Hkv, Hq // Hkv)).permute(0, 2, 3, 1, 4).reshape(B * Hkv, -1, D)
    kp, vp = (t[rk].float().transpose(1, 2).reshape(B * Hkv, mk, D) for t in (k, v))
    s = torch.bmm(qp, kp.transpose(1, 2).contiguous()).mul_(1 / math.sqrt(D)).view(B, Hkv, -1, mq, mk)
    seen = ik < lk[:, None, None]
    if st["causal"]:
        seen = seen & (ik <= (iq + (lk - lq)[:, None])[..., None])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    n = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(B * Hkv, -1, mk), vp).view(B, Hkv, -1, mq, D) / torch.where(n > 0, n, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, mq, Hq, D)
    return o[iq < lq[:, None]].to(q.dtype)


def _own_product(st):
    ss, c = _pkg(), st["case"]
    side = ss.SS_SPARSE_W if c["side"] == "W" else ss.SS_SPARSE_X
    return ss.spgemm_tiled_epilogue(side, c["M"], c["N"], st["dense"].shape[1], st["tv"], st["tm"], st["dense"], st["sx"],
                                    st["sw"], bias=st["bias"], act=c["act"], gated=c["gated"], residual=st["res"],
                                    y_dtype=st["y"])


def _own_rotary(st):
    return _pkg().rotary(st["x"], st["pos"], st["steps"], layout=st["layout"], mscale=st["mscale"])


def _own_attn(st):
    return _pkg().attn(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], k_len=st["k_len"], causal=st["causal"])


def run(st):
    op = st["case"]["op"]
    if own:
        return {"product": _own_product, "rotary": _own_rotary, "attn": _own_attn}[op](st)
    return {"product": _plain_product, "rotary": _plain_rotary, "attn": _plain_attn}[op](st)


# ---- the definitions in 64 bits ----------------------------------------------------------------------------


def _exact_product(c, st):
    z = torch.matmul(st["x"].double(), st["w"].double().t().contiguous())
    for s, shape in ((st["sx"], (-1, 1)), (st["sw"], (1, -1))):
        if s is not None:
            z *= s.double().view(shape)
    if st["bias"] is not None:
        z += st["bias"].double()

    def phi(t):
        if c["act"] == "relu":
            return torch.maximum(t, torch.zeros_like(t))
        if c["act"] == "silu":
            return t * torch.sigmoid(t)
        if c["act"] == "gelu":
            return t * torch.special.ndtr(t)
        if c["act"] == "gelu_tanh":
            return t * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))
        return t

    if c["gated"]:
        pair = z.view(c["M"], c["N"] // 2, 2)
        z = phi(pair[..., 0]) * pair[..., 1]
    else:
        z = phi(z)
    return z if st["res"] is None else z + st["res"].double()


def _exact_rotary(c, st):
    out = st["x"].double().clone()
    turn = torch.polar(torch.full((), float(st["mscale"]), dtype=torch.float64, device=DEV),
                       torch.outer(st["pos"].double(), st["freq"]))[:, None]
    n = c["rot"] // 2
    re, im = (slice(0, n), slice(n, 2 * n)) if c["layout"] == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    z = torch.complex(out[..., re], out[..., im]) * turn
    out[..., re], out[..., im] = z.real, z.imag
    return out


def _exact_attn(c, st):
    lq, lk, start = _lens(c)
    q, k, v = st["q"], st["k"], st["v"]
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    at = 0
    for a, b, s in zip(lq, lk, start):
        for h in range(c["Hkv"] if b else 0):
            x = q[at : at + a, h * G : (h + 1) * G].double().transpose(0, 1)
            score = (x @ k[s : s + b, h].double().t().contiguous()) / math.sqrt(c["D"])
            if c["causal"]:
                late = torch.ones((a, b), dtype=torch.bool, device=DEV).triu(b - a + 1)
                score = score.masked_fill(late, -math.inf)
            w = torch.softmax(score, -1).nan_to_num_(0.0)  # a row that sees no key: zeros
            out[at : at + a, h * G : (h + 1) * G] = (w @ v[s : s + b, h].double()).transpose(0, 1)
        at += a
    return out


def exact(c, seed):
    st = prepare(c, seed)
    return {"product": _exact_product, "rotary": _exact_rotary, "attn": _exact_attn}[c["op"]](c, st)
