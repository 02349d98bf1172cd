"""How the operators over groups of rows are called on the GPU: together, as an
expert layer and as adapters on a projection; their gradients; in captured graphs
and on other streams, two at once; with offsets and orders that are not what they
should be; with infinities and NaN in rows of other groups, magnitudes at the
types' ends and addresses past 2^31 values; and waits that run out.

Where results are compared for equality, inputs are small whole numbers, so that
every sum is exact in fp32 (test_gpu_groups.py)."""
import numpy as np
import pytest
import torch

from helpers import lib
from test_gpu_groups import TD, _code, _ints, _offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    return lib()


def _order(m, ids, groups):
    offsets = torch.empty(groups + 1, dtype=torch.int32, device="cuda")
    order, places = torch.empty_like(ids), torch.empty_like(ids)
    m.row_groups(ids, offsets, order, places)
    return offsets, order, places


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("tokens,dtype", [(1, "bf16"), (37, "f16"), (700, "bf16")])
def test_expert_layer(m, tokens, dtype):
    """Two of 12 experts for each token: order, products up and down, and back to the tokens with weights."""
    t, experts, top, hidden, inner = TD[dtype], 12, 2, 192, 320
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = (torch.randn(tokens, hidden, generator=g, device="cuda")).to(t)
    up, down = ((torch.randn(experts, *s, generator=g, device="cuda") * s[1] ** -0.5).to(t) for s in ((inner, hidden), (hidden, inner)))
    weights, ids = torch.softmax(torch.randn(tokens, experts, generator=g, device="cuda"), -1).topk(top)
    offsets, order, places = _order(m, ids.int().flatten(), experts)
    rows = x[order // top]
    h, y = torch.empty(tokens * top, inner, dtype=t, device="cuda"), torch.empty(tokens * top, hidden, dtype=t, device="cuda")
    m.GroupedGemm(experts, inner, hidden, dtype=_code(m, dtype)).run(rows, up, offsets, h)
    a = torch.nn.functional.silu(h.float()).to(t)
    m.GroupedGemm(experts, hidden, inner, dtype=_code(m, dtype)).run(a, down, offsets, y)
    out = (y[places.long()].view(tokens, top, hidden).double() * weights[..., None].double()).sum(1)
    want = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for i in range(tokens):
        for j in range(top):
            e = ids[i, j]
            hh = torch.nn.functional.silu(up[e].double() @ x[i].double())
            want[i] += weights[i, j].double() * (down[e].double() @ hh)
            size[i] += weights[i, j].double() * (down[e].double().abs() @ hh.abs())
    # h, a and y are rounded: at most half a step each of the products' magnitudes, and silu's slope is below 1.1
    # (h's own rounding is of its value: |h| and not |silu h|, which for negative h is up to |h| / |silu h| more,
    # but no more than 0.28 / 0.28 where the product counts; 4 half steps of sum |down| max(|a|, half |h|) hold it)
    big = torch.zeros_like(want)
    for i in range(tokens):
        for j in range(top):
            e = ids[i, j]
            big[i] += weights[i, j].double() * (down[e].double().abs() @ (up[e].double() @ x[i].double()).abs())
    assert ((out - want).abs() <= torch.finfo(t).eps / 2 * (1.2 * big + size + want.abs()) + 2.0**-18 * (size + big)).all()


@pytest.mark.parametrize("int4", [False, True])
def test_adapters_on_a_projection(m, int4):
    """The shared projection, dense or of int4 weights, and the adapters' change added in place."""
    rows, n, k, rank, groups = 24, 256, 512, 16, 6
    t = torch.float16
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, k, generator=g, device="cuda").to(t)
    y = torch.empty(rows, n, dtype=t, device="cuda")
    if int4:
        w = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        scales, zeros = torch.full((n, k // 128), 0.01, dtype=t, device="cuda"), torch.full((n, k // 128), 8.0, dtype=t, device="cuda")
        op = m.Gemm(m.make_desc(rows, n, k, a_dtype=m.GEMM_F16, b_dtype=m.GEMM_INT4, split_k=0, group_size=128))
        op.run(x, w, y, scales=scales, zeros=zeros)
    else:
        op = m.Gemm(m.make_desc(rows, n, k, a_dtype=m.GEMM_F16, split_k=0))
        op.run(x, (torch.randn(n, k, generator=g, device="cuda") * k**-0.5).to(t), y)
    shared = y.clone()
    a, b = (torch.randn(groups, rank, k, generator=g, device="cuda") * k**-0.5).to(t), (torch.randn(groups, n, rank, generator=g, device="cuda") * 0.3).to(t)
    ids = torch.randint(-1, groups, (rows,), generator=g, device="cuda", dtype=torch.int32)
    offsets, order, _ = _order(m, ids, groups)
    m.Adapters(groups, n, k, rank, dtype=m.GEMM_F16).run(x, a, b, offsets, order, y, y)
    for r, e in enumerate(ids.tolist()):
        if e < 0:
            assert torch.equal(y[r], shared[r])
            continue
        u = a[e].double() @ x[r].double()
        want = shared[r].double() + b[e].double() @ u
        off = 2.0**-20 * (a[e].double().abs() @ x[r].double().abs()) + 2.0**-16 * u.abs().max() + 2.0**-20 * u.abs()
        error = b[e].double().abs() @ off
        assert ((y[r].double() - want).abs() <= error + (want.abs() + error) * (2.0**-11 + 2.0**-23)).all()


def test_the_layer_example_runs():
    """It runs, and its gradients are those of the same layer in 64 bits (of its own choices of experts), but for the
    roundings of what lies between: half a step at each of six places of values that are sums of as many random signs,
    so 6 * 2^-8 of a gradient's norm is far beyond them and far below a wrong product's."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    layer = ex.ExpertLayer(128, 192, 8, 2, adapters=3, rank=8)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, d_out = (torch.randn(150, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    adapter = torch.randint(-1, 3, (150,), generator=g, device="cuda", dtype=torch.int32)
    out, kept = layer.forward(x, adapter)
    grads = layer.backward(kept, d_out)
    weights, ids = torch.softmax(x.float() @ layer.w_router.float().T, -1).topk(2)
    xd, up, down = (t.double().requires_grad_() for t in (x, layer.w_up, layer.w_down))
    mixed = torch.zeros(150, 128, dtype=torch.float64, device="cuda")
    for j in range(2):
        h = torch.einsum("th,tih->ti", xd, up[ids[:, j]])
        mixed = mixed + weights[:, j, None].double() * torch.einsum("ti,thi->th", torch.nn.functional.silu(h), down[ids[:, j]])
    want = torch.autograd.grad((mixed * d_out.double()).sum(), (xd, up, down))
    shared = x.double() @ layer.w_shared.double().T
    for r, e in enumerate(adapter.tolist()):
        if e >= 0:
            shared[r] += 2.0 * (layer.b[e].double() @ (layer.a[e].double() @ x[r].double()))
    for got, right in ((out, mixed.detach() + shared), *zip(grads, want)):
        assert float((got.double() - right).norm() / right.norm()) < 6 * 2.0**-8


def test_the_layer_example_without_adapter_numbers():
    """A layer that has adapters takes tokens without numbers as tokens of no adapter."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer_again", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    layer = ex.ExpertLayer(128, 192, 8, 2, adapters=3, rank=8)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(50, 128, generator=g, device="cuda").bfloat16()
    out, _ = layer.forward(x)
    same, _ = layer.forward(x, torch.full((50,), -1, dtype=torch.int32, device="cuda"))
    assert torch.equal(out, same)


# ------------------------------------------------------------------ gradients

@pytest.mark.parametrize("k_contig", [True, False])
@pytest.mark.parametrize("sizes", [[5, 0, 40, 1], [130, 300, 0, 77]], ids=["few", "many"])
def test_gradients(m, k_contig, sizes):
    """f = sum(C * dC): its gradients to A and B by the products, against the formula and against differences
    (f is linear in each, and whole numbers make both exact)."""
    t, n, k, groups, rows = torch.float16, 72, 136, len(sizes), sum(sizes)
    a, dc = _ints(1, rows, k, dtype=t), _ints(2, rows, n, dtype=t)
    b = _ints(3, groups, *((n, k) if k_contig else (k, n)), dtype=t)
    offsets, at = _offsets(sizes), np.concatenate([[0], np.cumsum(sizes)])
    layout, other = (m.GEMM_K_CONTIG, m.GEMM_MN_CONTIG) if k_contig else (m.GEMM_MN_CONTIG, m.GEMM_K_CONTIG)
    da, db = torch.empty_like(a), torch.empty_like(b)
    m.GroupedGemm(groups, k, n, b_layout=other, dtype=m.GEMM_F16).run(dc, b, offsets, da)
    op = m.GroupedGemmK(groups, *((n, k) if k_contig else (k, n)), dtype=m.GEMM_F16)
    op.run(*((dc, a) if k_contig else (a, dc)), offsets, db)
    for g in range(groups):
        lo, hi = at[g], at[g + 1]
        w = b[g].double() if k_contig else b[g].double().T
        assert torch.equal(da[lo:hi], (dc[lo:hi].double() @ w).to(t))
        want = dc[lo:hi].double().T @ a[lo:hi].double()
        assert torch.equal(db[g], (want if k_contig else want.T).to(t))

    forward = m.GroupedGemm(groups, n, k, b_layout=layout, dtype=m.GEMM_F16)

    def f(a, b):
        c = torch.zeros(rows, n, dtype=t, device="cuda")
        forward.run(a, b, offsets, c)
        return (c.double() * dc.double()).sum()
    for r, i in ((0, 0), (rows - 1, k - 1), (rows // 2, 77)):
        moved = a.clone()
        moved[r, i] += 1
        assert f(moved, b) - f(a, b) == da[r, i].double()
    for g in range(groups):
        for i, j in ((0, 0), (b.shape[1] - 1, b.shape[2] - 1)):
            moved = b.clone()
            moved[g, i, j] += 1
            assert f(a, moved) - f(a, b) == db[g, i, j].double()


@pytest.mark.parametrize("sizes", [[5, 0, 40, 1], [130, 300, 0, 77]], ids=["few", "many"])
@pytest.mark.parametrize("rank", [8, 48])
def test_adapter_gradients(m, sizes, rank):
    """The gradients through the adapters are products over groups: f = sum(out * dout), against the formula, and
    against differences of the adapters' own results.  Sums of at most 136 products of -1, 0
    and 1 are whole numbers that bf16 holds, those that may be larger are exact in fp32 and rounded once."""
    t, n, k, groups, rows = torch.bfloat16, 72, 136, len(sizes), sum(sizes)
    x, dout, base = (_ints(i, rows, c, dtype=t, most=1) for i, c in ((1, k), (2, n), (3, n)))
    a, b = _ints(4, groups, rank, k, dtype=t, most=1), _ints(5, groups, n, rank, dtype=t, most=1)
    offsets, at = _offsets(sizes), np.concatenate([[0], np.cumsum(sizes)])
    u, du, dx = (torch.empty(rows, c, dtype=t, device="cuda") for c in (rank, rank, k))
    da, db = torch.empty_like(a), torch.empty_like(b)
    m.GroupedGemm(groups, rank, k).run(x, a, offsets, u)
    m.GroupedGemm(groups, rank, n, b_layout=m.GEMM_MN_CONTIG).run(dout, b, offsets, du)
    m.GroupedGemm(groups, k, rank, b_layout=m.GEMM_MN_CONTIG).run(du, a, offsets, dx)
    m.GroupedGemmK(groups, rank, k).run(du, x, offsets, da)
    m.GroupedGemmK(groups, n, rank).run(dout, u, offsets, db)
    for g in range(groups):
        r = slice(at[g], at[g + 1])
        ud, dud = x[r].double() @ a[g].double().T, dout[r].double() @ b[g].double()
        assert torch.equal(u[r], ud.to(t)) and torch.equal(du[r], dud.to(t))
        assert torch.equal(dx[r], (dud @ a[g].double()).to(t))
        assert torch.equal(da[g], (dud.T @ x[r].double()).to(t)) and torch.equal(db[g], (dout[r].double().T @ ud).to(t))

    forward = m.Adapters(groups, n, k, rank)

    def f(x, a, b):
        out = torch.empty_like(base)
        forward.run(x, a, b, offsets, None, base, out)
        return out.double()
    # a step of one value of x: what it changes in its row is exact where bf16 holds both results, below 2^8
    for r, i in ((0, 0), (rows - 1, k - 1)):
        moved = x.clone()
        moved[r, i] += 1
        lo, hi = f(x, a, b)[r], f(moved, a, b)[r]
        exact = (lo.abs() < 256) & (hi.abs() < 256)
        g = next(j for j in range(groups) if at[j] <= r < at[j + 1])
        step = b[g].double() @ a[g, :, i].double()
        assert exact.any() and torch.equal((hi - lo)[exact], step[exact])
        assert dx[r, i] == (dout[r].double() @ step).to(t)


@pytest.mark.parametrize("sizes", [[5, 0, 40, 1], [130, 300, 0, 77]], ids=["few", "many"])
def test_adapter_gradients_by_differences(m, sizes):
    """f = sum(out * dout) moves by the gradients to x, A and B when one of their values moves by 1: f is linear in
    each.  With -1, 0 and 1 for all values, 8 of them in a sum and scales of 2, u is at most 9, what is added to base
    at most 2 * 8 * 9 (after the move), and out at most 145, which bf16 holds: all of it is exact."""
    t, n, k, rank, groups, rows = torch.bfloat16, 72, 8, 8, len(sizes), sum(sizes)
    x, dout, base = (_ints(i, rows, c, dtype=t, most=1) for i, c in ((1, k), (2, n), (3, n)))
    a, b = _ints(4, groups, rank, k, dtype=t, most=1), _ints(5, groups, n, rank, dtype=t, most=1)
    scales = torch.full((groups,), 2.0, device="cuda")
    offsets, at = _offsets(sizes), np.concatenate([[0], np.cumsum(sizes)])
    scaled = dout * 2
    u, du, dx = (torch.empty(rows, c, dtype=t, device="cuda") for c in (rank, rank, k))
    da, db = torch.empty_like(a), torch.empty_like(b)
    m.GroupedGemm(groups, rank, k).run(x, a, offsets, u)
    m.GroupedGemm(groups, rank, n, b_layout=m.GEMM_MN_CONTIG).run(scaled, b, offsets, du)
    m.GroupedGemm(groups, k, rank, b_layout=m.GEMM_MN_CONTIG).run(du, a, offsets, dx)
    m.GroupedGemmK(groups, rank, k).run(du, x, offsets, da)
    m.GroupedGemmK(groups, n, rank).run(scaled, u, offsets, db)
    forward = m.Adapters(groups, n, k, rank)

    def f(x, a, b):
        out = torch.empty_like(base)
        forward.run(x, a, b, offsets, None, base, out, scales=scales)
        return (out.double() * dout.double()).sum()

    def rounded(v):  # (the gradients are rounded once; their products' sums are whole numbers, which fp32 holds)
        return v.to(t)
    was = f(x, a, b)
    for r in (0, rows // 2, rows - 1):
        moved = x.clone()
        moved[r, r % k] += 1
        assert rounded(f(moved, a, b) - was) == dx[r, r % k]
    for g in range(groups):
        for i, j in ((0, 0), (3, 5), (rank - 1, k - 1)):
            moved = a.clone()
            moved[g, i, j] += 1
            assert rounded(f(x, moved, b) - was) == da[g, i, j], (g, i, j)
        for i, j in ((0, 0), (37, 2), (n - 1, rank - 1)):
            moved = b.clone()
            moved[g, i, j] += 1
            assert rounded(f(x, a, moved) - was) == db[g, i, j], (g, i, j)


# ------------------------------------------------------------------ graphs, streams, repeats

@pytest.mark.parametrize("kind", ["rows", "wide rows", "sums", "adapters", "adapters gathered", "adapters, two CTAs"])
def test_many_calls_one_after_the_other(m, kind, monkeypatch):
    """No wait runs out where copying warps have unequal work: narrow tiles of a plan for wider ones, tiles of few
    rows, many stages a tile.  (A warp that waits for stages that it brings nothing to can miss one.)"""
    g = torch.Generator(device="cuda").manual_seed(7)
    groups, n, k = (128, 1536, 2048) if "rows" in kind else (24, 520, 520) if kind == "sums" else (9, 512, 4096)
    per = 4 if kind == "rows" else 40 if "rows" in kind else 150 if kind == "sums" else 60
    rows = per * groups
    x, w = _ints(1, rows, k, dtype=torch.bfloat16), _ints(2, groups, n, k, dtype=torch.bfloat16)
    ids = [torch.randint(0, groups, (rows,), generator=g, device="cuda", dtype=torch.int32) for _ in range(4)]
    if kind == "adapters gathered":
        ids = [torch.where(torch.rand(rows, generator=g, device="cuda") < 0.03, i, i % 2 * 5) for i in ids]
    offsets, order, _ = zip(*(_order(m, i.int(), groups) for i in ids))
    if kind == "sums":
        op, outs = m.GroupedGemmK(groups, n, k), [torch.empty(groups, n, k, dtype=torch.bfloat16, device="cuda") for _ in ids]
        calls = [lambda i=i: op.run(x[:, :n], x, offsets[i], outs[i]) for i in range(4)]
    elif "rows" in kind:
        op, outs = m.GroupedGemm(groups, n, k), [torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda") for _ in ids]
        calls = [lambda i=i: op.run(x, w, offsets[i], outs[i]) for i in range(4)]
    else:
        monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", "2" if "two" in kind else "1")
        op, b = m.Adapters(groups, n, k, 16), _ints(3, groups, n, 16, dtype=torch.bfloat16, most=1)
        base, outs = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda"), [torch.empty(rows, n, dtype=torch.bfloat16, device="cuda") for _ in ids]
        a = _ints(4, groups, 16, k, dtype=torch.bfloat16, most=1)
        calls = [lambda i=i: op.run(x, a, b, offsets[i], order[i] if "gathered" in kind else None, base, outs[i]) for i in range(4)]
    for call in calls:
        call()
    assert op.sync_status() == m.GEMM_OK
    once = [o.clone() for o in outs]
    for i in range(400):
        calls[i % 4]()
    assert op.sync_status() == m.GEMM_OK
    assert all(torch.equal(o, p) for o, p in zip(once, outs))

def _operators(m, big):
    """Each operator on whole numbers: (its call, its output, what the output has to be for the present ids)."""
    t, groups, n, k, rank = torch.float16, 6, 264, 200, 16
    rows = 6000 if big else 50
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    offsets, order, places = torch.zeros(groups + 1, dtype=torch.int32, device="cuda"), torch.zeros_like(ids), torch.zeros_like(ids)
    a, b = _ints(1, rows, k, dtype=t), _ints(2, groups, n, k, dtype=t)
    c, d = torch.zeros(rows, n, dtype=t, device="cuda"), torch.zeros(groups, k, n, dtype=t, device="cuda")
    e = _ints(3, rows, n, dtype=t, most=1)
    down, up = _ints(4, groups, rank, k, dtype=t, most=1), _ints(5, groups, n, rank, dtype=t, most=1)
    out = torch.zeros_like(c)
    objects = m.GroupedGemm(groups, n, k, dtype=m.GEMM_F16), m.GroupedGemmK(groups, k, n, dtype=m.GEMM_F16), m.Adapters(groups, n, k, rank, dtype=m.GEMM_F16)

    def run(stream=None):
        m.row_groups(ids, offsets, order, places, stream=stream)
        objects[0].run(a, b, offsets, c, stream=stream)
        objects[1].run(a, e, offsets, d, stream=stream)
        objects[2].run(a, down, up, offsets, order, e, out, stream=stream)

    def check():
        assert all(o.sync_status() == m.GEMM_OK for o in objects)
        key = torch.where((ids < 0) | (ids >= groups), groups, ids).long()
        want = torch.sort(key, stable=True).indices
        assert torch.equal(order.long(), want)
        at = [int((key < g).sum()) for g in range(groups + 1)]
        assert offsets.tolist() == at
        wo = e.double()
        for g in range(groups):
            lo, hi = at[g], at[g + 1]
            assert torch.equal(c[lo:hi], (a[lo:hi].double() @ b[g].double().T).to(t))
            assert torch.equal(d[g], (a[lo:hi].double().T @ e[lo:hi].double()).to(t))
            r = want[lo:hi]
            wo[r] += (a[r].double() @ down[g].double().T) @ up[g].double().T
        assert torch.equal(out, wo.to(t))

    def draw(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ids.copy_(torch.randint(-1, groups, (rows,), generator=g, device="cuda"))
        if seed % 2:
            ids[ids == 2] = 3
    return run, check, draw, (c, d, out, order)


@pytest.mark.parametrize("big,form", [(False, ""), (True, ""), (True, "1"), (True, "2")])
def test_graph_replays_take_the_sizes_of_the_time(m, big, form, monkeypatch):
    monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", form)
    run, check, draw, _ = _operators(m, big)
    draw(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in range(1, 5):
        draw(seed)
        graph.replay()
        torch.cuda.synchronize()
        check()


@pytest.mark.parametrize("big,form", [(False, ""), (True, ""), (True, "1"), (True, "2")])
def test_streams(m, big, form, monkeypatch):
    """On a stream of the call's own, and two sets of operators at once on two streams."""
    monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", form)
    first, second = _operators(m, big), _operators(m, big)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for seed in range(3):
        first[2](seed)
        second[2](seed + 7)
        torch.cuda.synchronize()
        for _ in range(5):
            first[0](s1.cuda_stream)
            second[0](s2.cuda_stream)
        torch.cuda.synchronize()
        first[1]()
        second[1]()


@pytest.mark.parametrize("big", [False, True])
def test_one_object_on_two_streams(m, big):
    """Objects hold no workspace: runs of one may be under way at the same time."""
    t, n, k, sizes = torch.float16, 520, 264, [700, 0, 900, 41] if big else [3, 0, 9, 1]
    offsets = _offsets(sizes)
    op, opk = m.GroupedGemm(4, n, k, dtype=m.GEMM_F16), m.GroupedGemmK(4, k, n, dtype=m.GEMM_F16)
    sets = []
    for i in range(2):
        a, b, e = _ints(i, sum(sizes), k, dtype=t), _ints(i + 5, 4, n, k, dtype=t), _ints(i + 9, sum(sizes), n, dtype=t)
        sets.append((torch.cuda.Stream(), a, b, e, torch.empty(sum(sizes), n, dtype=t, device="cuda"), torch.empty(4, k, n, dtype=t, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, a, b, e, c, d in sets:
            op.run(a, b, offsets, c, stream=s.cuda_stream)
            opk.run(a, e, offsets, d, stream=s.cuda_stream)
    torch.cuda.synchronize()
    at = offsets.tolist()
    for _, a, b, e, c, d in sets:
        for g in range(4):
            lo, hi = at[g], at[g + 1]
            assert torch.equal(c[lo:hi], (a[lo:hi].double() @ b[g].double().T).to(t))
            assert torch.equal(d[g], (a[lo:hi].double().T @ e[lo:hi].double()).to(t))


@pytest.mark.parametrize("big,form", [(False, 0), (False, 8), (True, 0), (True, 1), (True, 2), (True, 4)])
def test_repeated_calls_give_the_same_bits(m, big, form, monkeypatch):
    monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", str(form))
    sizes = [2100, 0, 3111, 17] if big else [4, 0, 31, 1]
    rows, n, k, rank = sum(sizes), 520, 1000, 24
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*s):
        return torch.randn(s, generator=g, device="cuda").bfloat16()
    offsets, a, b, e, down, up = _offsets(sizes), normal(rows, k), normal(4, n, k), normal(rows, n), normal(4, rank, k), normal(4, n, rank)
    ops = m.GroupedGemm(4, n, k), m.GroupedGemmK(4, k, n), m.Adapters(4, n, k, rank)
    seen = []
    for _ in range(4):
        c, d, out = torch.empty(rows, n, dtype=a.dtype, device="cuda"), torch.empty(4, k, n, dtype=a.dtype, device="cuda"), torch.empty_like(e)
        ops[0].run(a, b, offsets, c)
        ops[1].run(a, e, offsets, d)
        ops[2].run(a, down, up, offsets, None, e, out)
        seen.append((c, d, out))
    for other in seen[1:]:
        assert all(torch.equal(x, y) for x, y in zip(seen[0], other))


# ------------------------------------------------------------------ offsets and orders

@pytest.mark.parametrize("offsets,means", [([0, 5, 3, 9], [0, 5, 5, 9]), ([-4, -1, 6, 60], [0, 0, 6, 20]), ([30, 40, 50, 60], [20, 20, 20, 20]),
                                           ([4, 4, 4, 4], [4, 4, 4, 4]), ([0, 2**31 - 1, -2**31, 7], [0, 20, 20, 20])])
def test_offsets_that_are_not_what_they_should_be(m, offsets, means):
    t, n, k, rank, rows = torch.float16, 72, 72, 8, 20
    at = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    a, b, e = _ints(1, rows, k, dtype=t), _ints(2, 3, n, k, dtype=t), _ints(3, rows, n, dtype=t)
    down, up = _ints(4, 3, rank, k, dtype=t, most=1), _ints(5, 3, n, rank, dtype=t, most=1)
    c, d, out = torch.full((rows, n), -7.0, dtype=t, device="cuda"), torch.empty(3, k, n, dtype=t, device="cuda"), torch.empty_like(e)
    m.GroupedGemm(3, n, k, dtype=m.GEMM_F16).run(a, b, at, c)
    m.GroupedGemmK(3, k, n, dtype=m.GEMM_F16).run(a, e, at, d)
    m.Adapters(3, n, k, rank, dtype=m.GEMM_F16).run(a, down, up, at, None, e, out)
    wc, wo = torch.full((rows, n), -7.0, dtype=torch.float64, device="cuda"), e.double()
    for g in range(3):
        lo, hi = means[g], means[g + 1]
        wc[lo:hi] = a[lo:hi].double() @ b[g].double().T
        assert torch.equal(d[g], (a[lo:hi].double().T @ e[lo:hi].double()).to(t))
        wo[lo:hi] += (a[lo:hi].double() @ down[g].double().T) @ up[g].double().T
    assert torch.equal(c, wc.to(t)) and torch.equal(out, wo.to(t))


@pytest.mark.parametrize("rows", [40, 6000])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("form", [0, 1, 2])
def test_order_with_numbers_of_no_row(m, rows, in_place, form, monkeypatch):
    """They are left out: their places' rows stay as they were."""
    monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", str(form))
    t, n, k, rank = torch.float16, 264, 136, 8
    order = torch.randperm(rows, device="cuda").int()
    gone = order[::7].clone()
    order[::7] = torch.tensor([-1, rows, 2**31 - 1, -2**31], dtype=torch.int32, device="cuda").repeat(rows)[:len(gone)]
    x, e = _ints(1, rows, k, dtype=t), _ints(2, rows, n, dtype=t)
    down, up = _ints(4, 2, rank, k, dtype=t, most=1), _ints(5, 2, n, rank, dtype=t, most=1)
    before = e.clone()
    out = e if in_place else torch.full_like(e, -9.0)
    sizes = [rows // 2, rows // 3]
    m.Adapters(2, n, k, rank, dtype=m.GEMM_F16).run(x, down, up, _offsets(sizes), order, e, out)
    want, at = before.double(), 0
    for g, size in enumerate(sizes):
        r = order[at:at + size].long()
        r = r[(r >= 0) & (r < rows)]
        want[r] += (x[r].double() @ down[g].double().T) @ up[g].double().T
        at += size
    if not in_place:
        want[gone.long()] = -9.0
    assert torch.equal(out, want.to(t))


# ------------------------------------------------------------------ infinities, NaN, magnitudes

@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("sizes", [[7, 3, 9, 0, 20], [200, 33, 150, 0, 300], [2000, 1100, 2500, 0, 600]], ids=["few", "some", "many"])
@pytest.mark.parametrize("form", [0, 1, 2])
def test_a_group_reaches_no_other(m, value, sizes, form, monkeypatch):
    """Group 1's rows, weights and adapter hold what is not finite; every other result is exact."""
    monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", str(form))
    t, n, k, rank, rows, groups = torch.float16, 264, 200, 24, sum(sizes), len(sizes)
    offsets, at = _offsets(sizes), np.concatenate([[0], np.cumsum(sizes)])
    lo1, hi1 = at[1], at[2]
    a, b, e = _ints(1, rows, k, dtype=t), _ints(2, groups, n, k, dtype=t), _ints(3, rows, n, dtype=t, most=1)
    down, up = _ints(4, groups, rank, k, dtype=t, most=1), _ints(5, groups, n, rank, dtype=t, most=1)
    for x in (a[lo1:hi1], e[lo1:hi1], b[1], down[1], up[1]):
        x.fill_(value)
    a[0, 3] = value  # and one row of group 0
    c, d, out = torch.zeros(rows, n, dtype=t, device="cuda"), torch.empty(groups, k, n, dtype=t, device="cuda"), torch.zeros(rows, n, dtype=t, device="cuda")
    m.GroupedGemm(groups, n, k, dtype=m.GEMM_F16).run(a, b, offsets, c)
    m.GroupedGemmK(groups, k, n, dtype=m.GEMM_F16).run(a, e, offsets, d)
    m.Adapters(groups, n, k, rank, dtype=m.GEMM_F16).run(a, down, up, offsets, None, e, out)
    for g in (0, 2, 3, 4):
        lo, hi = at[g] + (g == 0), at[g + 1]
        assert torch.equal(c[lo:hi], (a[lo:hi].double() @ b[g].double().T).to(t))
        assert torch.equal(out[lo:hi], (e[lo:hi].double() + (a[lo:hi].double() @ down[g].double().T) @ up[g].double().T).to(t))
        if g:
            assert torch.equal(d[g], (a[lo:hi].double().T @ e[lo:hi].double()).to(t))
    assert not c[lo1:hi1].isfinite().any() and not out[lo1:hi1].isfinite().any() and not d[1].isfinite().any() and not c[0].isfinite().all()
    col = torch.ones(k, dtype=torch.bool, device="cuda")
    col[3] = False
    assert torch.equal(d[0][col], (a[:lo1].double().T @ e[:lo1].double()).to(t)[col])


@pytest.mark.parametrize("rows,form", [(5, 0), (600, 0), (600, 1), (600, 2)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", ["large", "small"])
def test_adapters_between_magnitudes(m, rows, form, dtype, scale, monkeypatch):
    """A first product past the type's range, or below its least value, of a result that is neither."""
    monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", str(form))
    t, n, k, rank = TD[dtype], 264, 256, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    top = {"f16": {"large": (2.0**9, 2.0**9, 2.0**-14), "small": (2.0**-11, 2.0**-11, 2.0**12)},
           "bf16": {"large": (2.0**60, 2.0**60, 2.0**-120), "small": (2.0**-60, 2.0**-60, 2.0**118)}}[dtype][scale]
    x, a, b = ((torch.randn(s, generator=g, device="cuda") * v).to(t) for s, v in (((rows, k), top[0]), ((1, rank, k), top[1]), ((1, n, rank), top[2])))
    base, out = torch.zeros(rows, n, dtype=t, device="cuda"), torch.empty(rows, n, dtype=t, device="cuda")
    m.Adapters(1, n, k, rank, dtype=_code(m, dtype)).run(x, a, b, _offsets([rows]), None, base, out)
    u = x.double() @ a[0].double().T
    assert (u.abs().max() > 65504) if scale == "large" else (u.abs().max() < 2.0**-15)
    want = u @ b[0].double().T
    off = 2.0**-20 * (x.double().abs() @ a[0].double().abs().T) + 2.0**-16 * u.abs().amax(-1, keepdim=True) + 2.0**-20 * u.abs()
    error = off @ b[0].double().abs().T
    assert ((out.double() - want).abs() <= error + (want.abs() + error) * (torch.finfo(t).eps / 2 + 2.0**-23) + torch.finfo(t).smallest_normal * torch.finfo(t).eps).all()


# ------------------------------------------------------------------ far addresses

def test_rows_past_31_bits(m):
    """More than 2^31 values in A and C, and in B."""
    t, rows, n, k = torch.bfloat16, 150000, 16384, 64
    a, b = torch.zeros(rows, k, dtype=t, device="cuda"), _ints(2, 3, n, k, dtype=t)
    c = torch.zeros(rows, n, dtype=t, device="cuda")
    sizes = [140000, 3, 9000]
    marked = [0, 131071, 131072, 139999, 140001, 149002]
    for r in marked:
        a[r] = _ints(r, k, dtype=t)
    m.GroupedGemm(3, n, k).run(a, b, _offsets(sizes), c)
    for r in marked:
        g = 0 if r < 140000 else 1 if r < 140003 else 2
        assert torch.equal(c[r], (b[g].double() @ a[r].double()).to(t))
        a[r], c[r] = 0, 0
    assert not c.any()
    del a, b, c
    groups, n, k = 40, 8192, 8192
    a, b, c = _ints(1, 20, k, dtype=t), torch.zeros(groups, n, k, dtype=t, device="cuda"), torch.zeros(20, n, dtype=t, device="cuda")
    b[33, ::3], b[39, 1::2] = 1, 1
    sizes = [0] * groups
    sizes[33], sizes[39] = 12, 8
    m.GroupedGemm(groups, n, k).run(a, b, _offsets(sizes), c)
    want = torch.cat([a[:12].double() @ b[33].double().T, a[12:].double() @ b[39].double().T])
    assert torch.equal(c, want.to(t))


def test_sums_past_31_bits(m):
    t, groups, mm, n = torch.bfloat16, 40, 8192, 8192
    sizes = [0] * groups
    sizes[0], sizes[38], sizes[39] = 3, 20, 1
    a, b = _ints(1, 24, mm, dtype=t), _ints(2, 24, n, dtype=t)
    c = torch.ones(groups, mm, n, dtype=t, device="cuda")
    m.GroupedGemmK(groups, mm, n).run(a, b, _offsets(sizes), c)
    for g, lo, hi in ((0, 0, 3), (38, 3, 23), (39, 23, 24)):
        assert torch.equal(c[g], (a[lo:hi].float().T @ b[lo:hi].float()).to(t))
    assert not c[1:38].any()


@pytest.mark.parametrize("spread,form", [(False, 1), (False, 0), (False, 2), (True, 0)])
def test_adapters_past_31_bits(m, spread, form, monkeypatch):
    """More than 2^31 values in x and out, for few groups of many rows and for many of one row."""
    monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", str(form))
    t, rows, n, k, rank = torch.bfloat16, 36000, 65536, 65536, 8
    x, base = torch.zeros(rows, k, dtype=t, device="cuda"), torch.zeros(rows, n, dtype=t, device="cuda")
    groups = 2 if not spread else 5
    down, up = torch.zeros(groups, rank, k, dtype=t, device="cuda"), _ints(2, groups, n, rank, dtype=t)
    down[:, :, ::4096] = 1
    marked = [0, 32767, 32768, 35999]
    for r in marked:
        x[r, ::4096] = r % 5 + 1
    if spread:  # the marked rows alone, each with an adapter
        order = torch.tensor(marked, dtype=torch.int32, device="cuda")
        order = torch.cat([order, torch.tensor([r for r in range(rows) if r not in marked], dtype=torch.int32, device="cuda")])
        offsets = torch.tensor([0, 1, 2, 3, 4, 4], dtype=torch.int32, device="cuda")
    else:
        order, offsets = None, _offsets([34000, 2000])
    m.Adapters(groups, n, k, rank).run(x, down, up, offsets, order, base, base)
    for i, r in enumerate(marked):
        g = i if spread else int(r >= 34000)
        assert torch.equal(base[r], (up[g].double().sum(-1) * 16 * (r % 5 + 1)).to(t)), r
        base[r] = 0
    assert not base.any()


# ------------------------------------------------------------------ waits that run out

@pytest.mark.parametrize("kind", ["few rows", "few tiles", "many rows", "along K", "along K, narrow", "adapters 1", "adapters 2", "adapters 8"])
def test_waits_run_out(m, kind, monkeypatch):
    """A load that is withheld: the run's status says so, and the next run is right."""
    monkeypatch.setenv("LGT_GEMM_WAIT_LIMIT_MS", "20")
    t = torch.float16
    if kind in ("few rows", "few tiles", "many rows"):
        sizes, n, k = ([3, 9], 264, 200) if kind == "few rows" else ([3, 9], 264, 2000) if kind == "few tiles" else ([700, 400], 264, 200)
        a, b, c = _ints(1, sum(sizes), k, dtype=t), _ints(2, 2, n, k, dtype=t), torch.zeros(sum(sizes), n, dtype=t, device="cuda")
        op, args = m.GroupedGemm(2, n, k, dtype=m.GEMM_F16), (a, b, _offsets(sizes), c)
        want = torch.cat([a[:sizes[0]].double() @ b[0].double().T, a[sizes[0]:].double() @ b[1].double().T]).to(t)
        got, withhold = c, m._lib.gemm_grouped_withhold_load
    elif kind.startswith("along K"):
        n = 264 if kind == "along K" else 72
        a, b, c = _ints(1, 300, 200, dtype=t), _ints(2, 300, n, dtype=t), torch.zeros(2, 200, n, dtype=t, device="cuda")
        op, args = m.GroupedGemmK(2, 200, n, dtype=m.GEMM_F16), (a, b, _offsets([133, 167]), c)
        want = torch.stack([a[:133].double().T @ b[:133].double(), a[133:].double().T @ b[133:].double()]).to(t)
        got, withhold = c, m._lib.gemm_grouped_withhold_load
    else:
        monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", kind.split()[1])
        x, down, up, base = _ints(1, 900, 520, dtype=t), _ints(2, 1, 8, 520, dtype=t, most=1), _ints(3, 1, 1032, 8, dtype=t, most=1), _ints(4, 900, 1032, dtype=t)
        got = torch.zeros_like(base)
        op, args = m.Adapters(1, 1032, 520, 8, dtype=m.GEMM_F16), (x, down, up, _offsets([900]), None, base, got)
        want, withhold = (base.double() + (x.double() @ down[0].double().T) @ up[0].double().T).to(t), m._lib.gemm_adapters_withhold_load
    assert withhold(op.plan) == m.GEMM_OK
    op.run(*args)
    assert op.sync_status() == m.GEMM_ERR_TIMEOUT
    assert op.sync_status() == m.GEMM_OK
    op.run(*args)
    assert op.sync_status() == m.GEMM_OK and torch.equal(got, want)
