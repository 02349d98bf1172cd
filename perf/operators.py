"""The operators of one attention layer as it serves a language model, and the calls that are measured.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as a user calls the package:

  rope    per-head RMS norms of queries and keys with the position rotation in the same pass
  prompt  causal attention over packed prompts of different lengths, grouped heads
  cache   keys and values quantised to 8 bits as they are written into a paged cache, and read back
  decode  attention of one new token a sequence over that paged cache

`own` false: the plain forms; true: the package's entry points.
"""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3_MAX = 448.0


def listed():
    return [
        # 64 sequences, one new token each, a prompt length into a long context
        {"name": "rope_64tok_d128", "op": "rope", "tokens": 64, "hq": 32, "hk": 8, "d": 128, "rot": 128, "half": True, "norm": True, "dtype": "bf16", "base": 500000.0, "factor": 1.0, "context": 0, "start": 30000},
        # a batch of prompts, 16384 tokens in all
        {"name": "rope_16384tok_d128", "op": "rope", "tokens": 16384, "hq": 32, "hk": 8, "d": 128, "rot": 128, "half": True, "norm": True, "dtype": "bf16", "base": 500000.0, "factor": 1.0, "context": 0, "start": 0},
        # neighbouring pairs, half of each head turned, no norm, frequencies scaled for a context eight times the trained one; an odd token count
        {"name": "rope_4095tok_d64_part", "op": "rope", "tokens": 4095, "hq": 16, "hk": 16, "d": 64, "rot": 32, "half": False, "norm": False, "dtype": "f16", "base": 10000.0, "factor": 8.0, "context": 8192, "start": 50000},
        # four prompts of 4096 tokens, four query heads to a key head
        {"name": "prompt_4x4096_h32_8", "op": "prompt", "batch": 4, "longest": 4096, "spread": 0, "prefix": 0, "hq": 32, "hk": 8, "d": 128, "dtype": "bf16"},
        # one long prompt
        {"name": "prompt_1x16384_h16_2", "op": "prompt", "batch": 1, "longest": 16384, "spread": 0, "prefix": 0, "hq": 16, "hk": 2, "d": 128, "dtype": "bf16"},
        # thirteen prompts between 1 and 1999 tokens, odd group of three heads, head size 64
        {"name": "prompt_13ragged_h12_4_d64", "op": "prompt", "batch": 13, "longest": 1999, "spread": 7, "prefix": 0, "hq": 12, "hk": 4, "d": 64, "dtype": "f16"},
        # the next piece of prompts whose first 3000 tokens or so are there already
        {"name": "prompt_8x512_after_3000", "op": "prompt", "batch": 8, "longest": 512, "spread": 3, "prefix": 3000, "hq": 32, "hk": 8, "d": 128, "dtype": "bf16"},
        # one token each of 64 sequences into the cache
        {"name": "cache_64tok_h8_d128", "op": "cache", "tokens": 64, "hk": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # the prompts' tokens, all in one call
        {"name": "cache_16384tok_h8_d128", "op": "cache", "tokens": 16384, "hk": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # one user with a long context: few rows, a long axis
        {"name": "decode_1x65536_h32_8", "op": "decode", "batch": 1, "longest": 65536, "spread": 0, "hq": 32, "hk": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # 64 users of different lengths
        {"name": "decode_64ragged_8192_h32_8", "op": "decode", "batch": 64, "longest": 8192, "spread": 5, "hq": 32, "hk": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # a few short ones: latency counts; pages of 16, head size 64, six query heads to a key head
        {"name": "decode_5ragged_200_h12_2_d64", "op": "decode", "batch": 5, "longest": 200, "spread": 2, "hq": 12, "hk": 2, "d": 64, "page": 16, "dtype": "f16"},
    ]


def _log(rng, low, high):
    """A whole number between `low` and `high`, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("rope", "prompt", "cache", "decode"))
    d, dtype = rng.choice((64, 128)), rng.choice(("f16", "bf16"))
    hk = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 2, 3, 4, 6, 7, 8, 16))
    while hk * group > 48:
        group = rng.choice((1, 2, 4))
    if op == "rope":
        d = rng.choice((64, 96, 128, 256))
        scaled = rng.random() < 0.5
        tokens = max(1, min(_log(rng, 1, 16384), 16384 * 40 * 128 // (hk * (group + 1) * d)))
        return {"op": op, "tokens": tokens, "hq": hk * group, "hk": hk, "d": d, "rot": rng.choice((d, d, d // 2, 8 * rng.randint(1, d // 8))), "half": rng.random() < 0.6, "norm": rng.random() < 0.7, "dtype": dtype,
                "base": rng.choice((10000.0, 500000.0)), "factor": float(rng.choice((2, 4, 8))) if scaled else 1.0, "context": 8192 if scaled else 0, "start": rng.randint(0, 100000)}
    if op == "prompt":
        longest, prefix = _log(rng, 1, 8192), rng.choice((0, 0, _log(rng, 1, 4096)))
        batch = _log(rng, 1, 32)
        while batch > 1 and batch * hk * group * longest * (longest + prefix) > 1.5e9:
            batch = batch // 2
        while hk * group * longest * (longest + prefix) > 1.5e9:
            longest, prefix = longest // 2, prefix // 2
        return {"op": op, "batch": batch, "longest": max(1, longest), "spread": rng.choice((0, rng.randint(1, 999))), "prefix": prefix, "hq": hk * group, "hk": hk, "d": d, "dtype": dtype}
    if op == "cache":
        return {"op": op, "tokens": max(1, min(_log(rng, 1, 16384), 16384 * 8 * 128 // (hk * d))), "hk": hk, "d": d, "page": rng.choice((16, 32, 48, 64, 128)), "dtype": dtype}
    longest, batch = _log(rng, 1, 65536), _log(rng, 1, 256)
    while batch * longest * hk * d > 1 << 27:
        batch, longest = max(1, batch // 2), longest if batch > 1 else longest // 2
    return {"op": op, "batch": batch, "longest": longest, "spread": rng.choice((0, rng.randint(1, 999))), "hq": hk * group, "hk": hk, "d": d, "page": rng.choice((16, 32, 48, 64, 128)), "dtype": dtype}


def _lengths(case, lowest=1):
    """Lengths of the case's sequences: all the longest, or spread evenly in their logarithm with the longest among them."""
    if not case["spread"]:
        return [case["longest"]] * case["batch"]
    r = random.Random(case["spread"])
    return [case["longest"]] + [max(lowest, _log(r, 1, case["longest"])) for _ in range(case["batch"] - 1)]


def _prefixes(case):
    """How many keys each sequence has before its first query."""
    r = random.Random(case["spread"] + 1)
    return [r.randint(max(1, case["prefix"] // 2), case["prefix"]) if case["prefix"] else 0 for _ in range(case["batch"])]


def _frequencies(case):
    """Radians a position for each pair. Pairs that turn fewer than once in the trained context are slowed by `factor`, those that turn over 4 times are kept, those between are blended."""
    f = case["base"] ** (-torch.arange(case["rot"] // 2, dtype=torch.float64) * 2 / case["rot"])
    if case["factor"] == 1.0:
        return f
    keep = ((case["context"] * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
    return f * (keep + (1 - keep) / case["factor"])


def _cumulative(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _handle(case):
    """What a program that uses the package makes once and keeps."""
    if not own:
        return None
    import layout_general_tensor_gb300 as lgt

    dtype = lgt.GEMM_BF16 if case["dtype"] == "bf16" else lgt.GEMM_F16
    if case["op"] == "rope":
        return lgt.QKNormRope(case["hq"], case["hk"], case["d"], rot_dim=case["rot"], layout=lgt.ATTN_ROPE_HALF if case["half"] else lgt.ATTN_ROPE_INTERLEAVED, dtype=dtype, eps=1e-6, base=case["base"],
                              factor=case["factor"], context=case["context"], low_turns=1.0, high_turns=4.0)
    if case["op"] == "prompt":
        return lgt.PromptAttention(case["hq"], case["hk"], case["d"], dtype=dtype, causal=True)
    if case["op"] == "decode":
        return lgt.CacheAttention(case["hq"], case["hk"], case["d"], case["page"], dtype=dtype)
    return None


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype, d, hk = DT[case["dtype"]], case["d"], case["hk"]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case, "handle": _handle(case)}
    if case["op"] == "rope":
        t, hq = case["tokens"], case["hq"]
        s["qkv"] = normal(t, (hq + 2 * hk) * d, scale=2.0)  # as the projection leaves it
        s["q"], s["k"] = s["qkv"][:, : hq * d].view(t, hq, d), s["qkv"][:, hq * d : (hq + hk) * d].view(t, hk, d)
        s["wq"], s["wk"] = (normal(d, scale=0.1) + 1, normal(d, scale=0.1) + 1) if case["norm"] else (None, None)
        s["positions"] = (torch.arange(t, device="cuda", dtype=torch.int32) * 7 % 30011) + case["start"]
        s["frequencies"] = _frequencies(case).to("cuda", torch.float32)
        s["q_out"], s["k_out"] = torch.empty(t, hq, d, dtype=dtype, device="cuda"), torch.empty(t, hk, d, dtype=dtype, device="cuda")
    elif case["op"] == "prompt":
        nq = _lengths(case)
        nk = [a + b for a, b in zip(nq, _prefixes(case))]
        s["q"], s["k"], s["v"] = normal(sum(nq), case["hq"], d), normal(sum(nk), hk, d), normal(sum(nk), hk, d)
        s["cu_q"], s["cu_k"], s["most_q"], s["most_k"] = _cumulative(nq), _cumulative(nk), max(nq), max(nk)
        s["out"] = torch.empty(sum(nq), case["hq"], d, dtype=dtype, device="cuda")
    elif case["op"] == "cache":
        t, page = case["tokens"], case["page"]
        pages = -(-t // page) + 3
        s["k"], s["v"] = normal(t, hk, d), normal(t, hk, d, scale=0.3)
        order = torch.randperm(pages, generator=g, device="cuda")  # pages as an allocator hands them out
        at = torch.arange(t, device="cuda")
        s["slots"] = (order[at // page] * page + at % page).to(torch.int32)
        s["cache"] = _empty_cache(pages, page, hk, d)
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        s["handle"] = _package_cache(s["cache"])
    else:
        n, page = _lengths(case), case["page"]
        most = -(-max(n) // page)
        pages = sum(-(-x // page) for x in n)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        s["table"] = torch.zeros(len(n), most, dtype=torch.int32, device="cuda")
        used = 0
        for b, x in enumerate(n):
            s["table"][b, : -(-x // page)] = order[used : used + -(-x // page)]
            used += -(-x // page)
        s["lengths"] = torch.tensor(n, dtype=torch.int32, device="cuda")
        s["q"] = normal(len(n), case["hq"], d)
        s["cache"] = _empty_cache(pages, page, hk, d)
        for name, scale in (("k", 1.0), ("v", 0.3)):
            step = max(1, (1 << 26) // (hk * page * d))
            for p in range(0, pages, step):
                x = torch.randn((min(step, pages - p), hk, page, d), generator=g, device="cuda") * scale
                s["cache"][name][p : p + step], s["cache"][name + "_exp"][p : p + step] = _quantise(x)
        s["out"] = torch.empty_like(s["q"])
        s["package_cache"] = _package_cache(s["cache"])
    return s


def _empty_cache(pages, page, hk, d):
    """The cache: 8-bit codes [page][head][token][d], and a power of two for each [page][head][token], held as its exponent + 127."""
    made = {n: torch.zeros(pages, hk, page, d, dtype=torch.uint8, device="cuda") for n in ("k", "v")}
    made.update({n + "_exp": torch.zeros(pages, hk, page, dtype=torch.uint8, device="cuda") for n in ("k", "v")})
    return made


def _package_cache(cache):
    if not own:
        return None
    import layout_general_tensor_gb300 as lgt

    return lgt.KVCache(cache["k"], cache["v"], cache["k_exp"], cache["v_exp"])


def _quantise(x):
    """Rows of x (32 bits) as e4m3 codes and the smallest power of two that keeps the row within e4m3's range."""
    part, power = torch.frexp(x.abs().amax(-1))  # amax = part * 2^power, part in [0.5, 1); 448 = 0.875 * 2^9
    power = torch.where(part == 0, torch.zeros_like(power), power - 9 + (part > 0.875)).clamp(-126, 127)
    codes = torch.ldexp(x, -power[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (power + 127).to(torch.uint8)


def _values(codes, exponents):
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), exponents[..., None].int() - 127)


def _plain_rope(s):
    case, rot = s["case"], s["case"]["rot"]
    angle = s["positions"].float()[:, None, None] * s["frequencies"]
    cos, sin = torch.cos(angle), torch.sin(angle)

    def turn(x, weight):
        y = x.float()
        if weight is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.float()
        r = y[..., :rot]
        a, b = (r[..., : rot // 2], r[..., rot // 2 :]) if case["half"] else (r[..., 0::2], r[..., 1::2])
        c, e = a * cos - b * sin, b * cos + a * sin
        r = torch.cat((c, e), -1) if case["half"] else torch.stack((c, e), -1).flatten(-2)
        return torch.cat((r, y[..., rot:]), -1).to(x.dtype)

    return {"q": turn(s["q"], s["wq"]), "k": turn(s["k"], s["wk"])}


def _softmax(scores, visible):
    """Rows' weights over the keys that they see; a row that sees none has none."""
    scores = scores.masked_fill(~visible, -math.inf)
    most = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(most == -math.inf, torch.zeros_like(most), most))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _plain_prompt(s):
    case, q, k, v = s["case"], s["q"], s["k"], s["v"]
    hq, hk, d = case["hq"], case["hk"], case["d"]
    nq, nk = (c[1:] - c[:-1] for c in (s["cu_q"], s["cu_k"]))
    iq, ik = torch.arange(s["most_q"], device="cuda"), torch.arange(s["most_k"], device="cuda")

    def padded(x, cu, i):  # [sequence, head, token, d]; what is past a sequence's end is not used
        return x.float()[(cu[:-1, None] + i).clamp(max=x.shape[0] - 1)].transpose(1, 2)

    queries = padded(q, s["cu_q"], iq).reshape(case["batch"], hk, hq // hk * s["most_q"], d)
    keys, values = padded(k, s["cu_k"], ik), padded(v, s["cu_k"], ik)
    scores = (queries @ keys.transpose(2, 3)).view(case["batch"], hq, s["most_q"], s["most_k"]) * (1 / math.sqrt(d))
    visible = ik <= (iq[:, None] + (nk - nq)[:, None, None])  # the last query sees the last key
    weights = _softmax(scores, (visible & (ik < nk[:, None, None]))[:, None])
    out = (weights.view(case["batch"], hk, -1, s["most_k"]) @ values).view(case["batch"], hq, s["most_q"], d).transpose(1, 2)
    row = torch.arange(q.shape[0], device="cuda")
    b = torch.searchsorted(s["cu_q"][1:].contiguous(), row.int(), right=True)
    return out[b, row - s["cu_q"][b]].to(q.dtype)


def _plain_cache(s):
    c, slots = s["cache"], s["slots"].long()
    page = s["case"]["page"]
    at, off = slots // page, slots % page
    for name in ("k", "v"):
        c[name][at, :, off], c[name + "_exp"][at, :, off] = _quantise(s[name].float())
    most = torch.finfo(s["k"].dtype).max
    return {n: _values(c[n][at, :, off], c[n + "_exp"][at, :, off]).clamp(-most, most).to(s["k"].dtype) for n in ("k", "v")}


def _plain_decode(s):
    case, c, table = s["case"], s["cache"], s["table"].long()
    b, hq, d = s["q"].shape
    hk = case["hk"]
    keys, values = (_values(c[n][table], c[n + "_exp"][table]).transpose(1, 2).reshape(b, hk, -1, d) for n in ("k", "v"))
    scores = (s["q"].float().view(b, hk, hq // hk, d) @ keys.transpose(2, 3)) * (1 / math.sqrt(d))
    weights = _softmax(scores, (torch.arange(keys.shape[2], device="cuda") < s["lengths"][:, None])[:, None, None])
    return (weights @ values).view(b, hq, d).to(s["q"].dtype)


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "prompt": _plain_prompt, "cache": _plain_cache, "decode": _plain_decode}[op](s)
    if op == "rope":
        s["handle"].run(s["q"], s["k"], s["positions"], s["q_out"], s["k_out"], s["wq"], s["wk"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "prompt":
        s["handle"].run(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"])
        return s["out"]
    if op == "cache":
        s["handle"].write(s["k"], s["v"], s["slots"])
        s["handle"].read(s["slots"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    s["handle"].run(s["q"], s["package_cache"], s["table"], s["lengths"], s["out"])
    return s["out"]


def work(case):
    hk, d = case["hk"], case["d"]
    if case["op"] == "rope":
        n = case["tokens"] * (case["hq"] + hk) * d
        return {"bytes": 4 * n + 4 * case["tokens"] + (4 * d if case["norm"] else 0), "flops": (7 if case["norm"] else 3) * n}
    if case["op"] == "prompt":
        nq, before = _lengths(case), _prefixes(case)
        seen = sum(n * p + n * (n + 1) // 2 for n, p in zip(nq, before))
        return {"bytes": 2 * d * (2 * case["hq"] * sum(nq) + 2 * hk * sum(map(sum, zip(nq, before)))), "flops": 4 * case["hq"] * d * seen}
    if case["op"] == "cache":  # in and out at 16 bits, the codes written and read, the exponents too
        return {"bytes": 2 * case["tokens"] * hk * (2 * d + d + 1 + d + 1 + 2 * d) + 8 * case["tokens"], "flops": 6 * case["tokens"] * hk * d}
    n = _lengths(case)
    return {"bytes": 2 * sum(n) * hk * (d + 1) + 4 * case["batch"] * case["hq"] * d + 4 * sum(-(-x // case["page"]) for x in n) + 4 * len(n), "flops": 4 * case["hq"] * d * sum(n)}


# From here on: the operators' definitions in 64 bits, sequence by sequence and head by head.


def _e4m3_row(x):
    """x in 64 bits, each row on the e4m3 grid times the least power of two >= amax / 448."""
    most = x.abs().amax(-1, keepdim=True)
    step = torch.where(most > 0, torch.exp2(torch.ceil(torch.log2(most / E4M3_MAX))), torch.ones_like(most))
    y = x / step
    grid = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)  # three bits after the leading one, least exponent -6
    return torch.round(y / grid) * grid * step


def exact(case, seed):
    s = prepare(case, seed)
    d, hk = case["d"], case["hk"]
    if case["op"] == "rope":
        phase = torch.outer(s["positions"].double(), _frequencies(case).to("cuda"))
        z, found = torch.polar(torch.ones_like(phase), phase), {}
        for name, weight in (("q", s["wq"]), ("k", s["wk"])):
            y = s[name].double()
            if weight is not None:
                y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.double()
            i = torch.arange(case["rot"] // 2, device="cuda")
            a, b = (i, i + case["rot"] // 2) if case["half"] else (2 * i, 2 * i + 1)
            turned = torch.complex(y[..., a], y[..., b]) * z[:, None]
            y = y.clone()
            y[..., a], y[..., b] = turned.real, turned.imag
            found[name] = y
        return found
    if case["op"] == "cache":
        most = torch.finfo(s["k"].dtype).max
        return {n: _e4m3_row(s[n].double()).clamp(-most, most) for n in ("k", "v")}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["hq"] // hk
    if case["op"] == "prompt":
        cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
        for b in range(case["batch"]):
            q, k, v = s["q"][cu_q[b] : cu_q[b + 1]].double(), s["k"][cu_k[b] : cu_k[b + 1]].double(), s["v"][cu_k[b] : cu_k[b + 1]].double()
            hidden = torch.triu(torch.ones(len(q), len(k), dtype=torch.bool, device="cuda"), len(k) - len(q) + 1)
            for h in range(case["hq"]):
                logits = (q[:, h] @ k[:, h // group].T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
                out[cu_q[b] : cu_q[b + 1], h] = torch.softmax(logits, -1) @ v[:, h // group]
        return out
    c, table = s["cache"], s["table"]
    for b, n in enumerate(_lengths(case)):
        at = torch.arange(n, device="cuda")
        at, off = table[b].long()[at // case["page"]], at % case["page"]
        k, v = (c[x][at, :, off].view(torch.float8_e4m3fn).double() * torch.exp2(c[x + "_exp"][at, :, off].double() - 127)[..., None] for x in ("k", "v"))
        for h in range(hk):
            rows = slice(h * group, (h + 1) * group)
            out[b, rows] = torch.softmax(s["q"][b, rows].double() @ k[:, h].T / math.sqrt(d), -1) @ v[:, h]
    return out
