"""Products whose weights differ from row to row, and the calls that are measured.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as a user calls the package:

  groups    rows put in order by the group that each belongs to: offsets, order and places from group numbers
  rows      products grouped by expert: every group of rows times a matrix of its own
  sums      the gradient to those matrices: for every group, the product of two tensors over the group's rows
  adapters  low-rank adapters of many requests at once, added to a shared projection

`own` false: the plain forms; true: the package's entry points.
"""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # 64 new tokens, eight experts each: latency
        {"name": "groups_512_of_128", "op": "groups", "rows": 512, "groups": 128, "none": 0.0, "spread": 1},
        # a batch of prompts, 16384 tokens with eight experts each; some belong to another device's experts
        {"name": "groups_131072_of_128", "op": "groups", "rows": 131072, "groups": 128, "none": 0.1, "spread": 2},
        # one new token through eight of 64 experts, the weights as a gradient pass or an untransposed checkpoint has them
        {"name": "rows_8_of_64", "op": "rows", "rows": 8, "pad": 0, "groups": 64, "n": 2048, "k": 4096, "k_contig": False, "dtype": "bf16", "spread": 3},
        # 64 new tokens through eight of 128 experts: every expert's weights, a few rows each
        {"name": "rows_512_of_128", "op": "rows", "rows": 512, "pad": 0, "groups": 128, "n": 1536, "k": 2048, "k_contig": True, "dtype": "bf16", "spread": 4},
        # prompts: about a thousand rows an expert
        {"name": "rows_16384_of_16", "op": "rows", "rows": 16384, "pad": 0, "groups": 16, "n": 4096, "k": 4096, "k_contig": True, "dtype": "bf16", "spread": 5},
        # odd sizes, a padded batch
        {"name": "rows_4000_of_24_padded", "op": "rows", "rows": 4000, "pad": 95, "groups": 24, "n": 3000, "k": 2880, "k_contig": False, "dtype": "f16", "spread": 6},
        # the weights' gradient of a training step
        {"name": "sums_16384_of_16", "op": "sums", "rows": 16384, "pad": 0, "groups": 16, "m": 2048, "n": 4096, "dtype": "bf16", "spread": 7},
        # few rows an expert, some experts without any: what is written is most of the work
        {"name": "sums_1001_of_40", "op": "sums", "rows": 1001, "pad": 23, "groups": 40, "m": 1000, "n": 2880, "dtype": "f16", "spread": 8},
        # one user's new token
        {"name": "adapters_1_of_4_r8", "op": "adapters", "rows": 1, "none": 0, "groups": 4, "n": 1024, "k": 4096, "rank": 8, "sorted": False, "dtype": "f16", "spread": 9},
        # one new token each of 64 users, most with an adapter of their own
        {"name": "adapters_64_of_100_r16", "op": "adapters", "rows": 60, "none": 4, "groups": 100, "n": 4096, "k": 4096, "rank": 16, "sorted": False, "dtype": "bf16", "spread": 10},
        # odd sizes, prompts and new tokens mixed, some requests without an adapter
        {"name": "adapters_999_of_13_r24", "op": "adapters", "rows": 801, "none": 198, "groups": 13, "n": 3000, "k": 2880, "rank": 24, "sorted": False, "dtype": "f16", "spread": 11},
        # prompts, one request after the other
        {"name": "adapters_16384_of_8_r64", "op": "adapters", "rows": 16384, "none": 0, "groups": 8, "n": 4096, "k": 4096, "rank": 64, "sorted": True, "dtype": "bf16", "spread": 12},
    ]


def _log(rng, low, high):
    """A whole number between `low` and `high`, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op, dtype, spread = rng.choice(("groups", "rows", "sums", "adapters")), rng.choice(("f16", "bf16")), rng.randint(100, 1 << 30)
    if op == "groups":
        return {"op": op, "rows": _log(rng, 1, 131072), "groups": _log(rng, 1, 512), "none": rng.choice((0.0, 0.3 * rng.random())), "spread": spread}
    if op == "adapters":
        rows, n, k = _log(rng, 1, 16384), 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 1024)
        while rows * (2 * n + k) > 16384 * 12288:
            n, k = max(64, n // 16 * 8), max(64, k // 16 * 8)
        return {"op": op, "rows": rows, "none": rng.choice((0, rng.randint(0, rows))) if rows < 8192 else 0, "groups": _log(rng, 1, 128), "n": n, "k": k, "rank": 8 * rng.choice((1, 2, 2, 3, 4, 8, 8, 11, 16)),
                "sorted": rng.random() < 0.3, "dtype": dtype, "spread": spread}
    rows, groups, a, b = _log(rng, 1, 32768), _log(rng, 1, 128), 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 1024)
    while groups * a * b > 4e8 or rows * a * b > 2.5e11:
        a, b, groups = max(64, a // 16 * 8), max(64, b // 16 * 8), max(1, groups * 3 // 4)
    made = {"op": op, "rows": rows, "pad": rng.choice((0, rng.randint(1, 200))), "groups": groups, "n": a, "dtype": dtype, "spread": spread}
    return {**made, "k": b, "k_contig": rng.random() < 0.5} if op == "rows" else {**made, "m": b}


def _sizes(case):
    """How many rows each group has: some groups are chosen several times as often as others, and of few rows many groups have none."""
    r, sizes = random.Random(case["spread"]), [0] * case["groups"]
    for g in r.choices(range(case["groups"]), [math.exp(r.gauss(0, 0.7)) for _ in sizes], k=case["rows"]):
        sizes[g] += 1
    return sizes


def _cumulative(sizes):
    at = [0]
    for n in sizes:
        at.append(at[-1] + n)
    return at


def _handle(case):
    """What a program that uses the package makes once and keeps."""
    if not own or case["op"] == "groups":
        return None
    import layout_general_tensor_gb300 as lgt

    dtype = lgt.GEMM_BF16 if case["dtype"] == "bf16" else lgt.GEMM_F16
    if case["op"] == "rows":
        return lgt.GroupedGemm(case["groups"], case["n"], case["k"], b_layout=lgt.GEMM_K_CONTIG if case["k_contig"] else lgt.GEMM_MN_CONTIG, dtype=dtype)
    if case["op"] == "sums":
        return lgt.GroupedGemmK(case["groups"], case["m"], case["n"], dtype=dtype)
    return lgt.Adapters(case["groups"], case["n"], case["k"], case["rank"], dtype=dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "handle": _handle(case)}
    if case["op"] == "groups":
        r, most = random.Random(case["spread"]), case["groups"]
        liked = torch.tensor([math.exp(r.gauss(0, 0.7)) for _ in range(most)], device="cuda")
        s["ids"] = torch.multinomial(liked, case["rows"], replacement=True, generator=g).to(torch.int32)
        s["ids"][torch.rand(case["rows"], generator=g, device="cuda") < case["none"]] = -1  # of no group here
        s["offsets"] = torch.empty(most + 1, dtype=torch.int32, device="cuda")
        s["order"], s["places"] = (torch.empty(case["rows"], dtype=torch.int32, device="cuda") for _ in range(2))
        return s
    dtype, rows = DT[case["dtype"]], case["rows"]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)

    s["at"] = _cumulative(_sizes(case))
    s["offsets"] = torch.tensor(s["at"], dtype=torch.int32, device="cuda")
    if case["op"] == "rows":
        n, k, all_rows = case["n"], case["k"], rows + case["pad"]
        s["a"] = normal(all_rows, k)
        s["b"] = normal(case["groups"], *((n, k) if case["k_contig"] else (k, n)), scale=1 / math.sqrt(k))
        s["out"] = torch.zeros(all_rows, n, dtype=dtype, device="cuda")
    elif case["op"] == "sums":
        s["a"], s["b"] = normal(rows + case["pad"], case["m"]), normal(rows + case["pad"], case["n"], scale=0.02)
        s["out"] = torch.empty(case["groups"], case["m"], case["n"], dtype=dtype, device="cuda")
    else:
        n, k, rank, all_rows = case["n"], case["k"], case["rank"], rows + case["none"]
        s["x"], s["base"] = normal(all_rows, k), normal(all_rows, n)
        s["down"], s["up"] = normal(case["groups"], rank, k, scale=1 / math.sqrt(k)), normal(case["groups"], n, rank, scale=0.1)
        s["scales"] = torch.rand(case["groups"], generator=g, device="cuda") + 0.5
        s["order"] = None if case["sorted"] else torch.randperm(all_rows, generator=g, device="cuda").to(torch.int32)
        s["out"] = torch.empty_like(s["base"])
    return s


def _plain_groups(s):
    ids, most = s["ids"].long(), s["case"]["groups"]
    key = torch.where((ids < 0) | (ids >= most), most, ids)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(most + 1, dtype=torch.int64, device="cuda").index_add_(0, key, torch.ones_like(key))
    s["order"].copy_(order)
    s["places"][order] = torch.arange(len(ids), dtype=torch.int32, device="cuda")
    s["offsets"].copy_(torch.cumsum(counts, 0) - counts)
    return {"offsets": s["offsets"], "order": s["order"], "places": s["places"]}


def _plain_rows(s):
    for e, (low, high) in enumerate(zip(s["at"], s["at"][1:])):
        if high > low:
            b = s["b"][e].float()
            s["out"][low:high] = (s["a"][low:high].float() @ (b.T if s["case"]["k_contig"] else b)).to(s["out"].dtype)
    return s["out"]


def _plain_sums(s):
    for e, (low, high) in enumerate(zip(s["at"], s["at"][1:])):
        s["out"][e] = (s["a"][low:high].float().T @ s["b"][low:high].float()).to(s["out"].dtype)
    return s["out"]


def _plain_adapters(s):
    case, out = s["case"], s["out"]
    out.copy_(s["base"])
    for e, (low, high) in enumerate(zip(s["at"], s["at"][1:])):
        if high > low:
            at = slice(low, high) if case["sorted"] else s["order"][low:high].long()
            change = (s["x"][at].float() @ s["down"][e].float().T) @ s["up"][e].float().T
            out[at] = (s["base"][at].float() + s["scales"][e] * change).to(out.dtype)
    return out


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"groups": _plain_groups, "rows": _plain_rows, "sums": _plain_sums, "adapters": _plain_adapters}[op](s)
    if op == "groups":
        import layout_general_tensor_gb300 as lgt

        lgt.row_groups(s["ids"], s["offsets"], s["order"], s["places"])
        return {"offsets": s["offsets"], "order": s["order"], "places": s["places"]}
    if op == "adapters":
        s["handle"].run(s["x"], s["down"], s["up"], s["offsets"], s["order"], s["base"], s["out"], scales=s["scales"])
    else:
        s["handle"].run(s["a"], s["b"], s["offsets"], s["out"])
    return s["out"]


def work(case):
    if case["op"] == "groups":
        return {"bytes": 12 * case["rows"] + 4 * case["groups"] + 4, "flops": 2 * case["rows"]}
    sizes, rows = _sizes(case), case["rows"]
    table, active = 4 * len(sizes) + 4, sum(n > 0 for n in sizes)
    if case["op"] == "rows":
        n, k = case["n"], case["k"]
        return {"bytes": table + 2 * rows * (n + k) + 2 * active * n * k, "flops": 2 * rows * n * k}
    if case["op"] == "sums":
        return {"bytes": table + 2 * rows * (case["m"] + case["n"]) + 2 * len(sizes) * case["m"] * case["n"], "flops": 2 * rows * case["m"] * case["n"]}
    n, k, rank, none = case["n"], case["k"], case["rank"], case["none"]
    return {"bytes": table + 4 * active + 2 * rows * (k + 2 * n) + 4 * none * n + 2 * active * rank * (n + k) + (0 if case["sorted"] else 4 * (rows + none)), "flops": 2 * rows * rank * (n + k)}


# From here on: the operators' definitions in 64 bits, group by group.


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "groups":
        ids, most = s["ids"].tolist(), case["groups"]
        members = [[] for _ in range(most + 1)]
        for r, e in enumerate(ids):
            members[e if 0 <= e < most else most].append(r)
        order = [r for m in members for r in m]
        places = [0] * len(order)
        for i, r in enumerate(order):
            places[r] = i
        return {n: torch.tensor(v, dtype=torch.int32, device="cuda") for n, v in (("offsets", _cumulative([len(m) for m in members[:most]])), ("order", order), ("places", places))}
    found = s["base"].double() if case["op"] == "adapters" else torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["groups"]):
        low, high = s["at"][e], s["at"][e + 1]
        if low == high:
            continue
        if case["op"] == "rows":
            found[low:high] = torch.einsum("rk,nk->rn" if case["k_contig"] else "rk,kn->rn", s["a"][low:high].double(), s["b"][e].double())
        elif case["op"] == "sums":
            found[e] = torch.einsum("rm,rn->mn", s["a"][low:high].double(), s["b"][low:high].double())
        else:
            r = torch.arange(low, high, device="cuda") if case["sorted"] else s["order"][low:high].long()
            found[r] += torch.einsum("rk,jk,nj->rn", s["x"][r].double(), s["down"][e].double(), s["up"][e].double()) * s["scales"][e].double()
    return found
