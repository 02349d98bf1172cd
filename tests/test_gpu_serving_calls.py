"""How the serving operators are called on the GPU: captured in a graph, with
workspaces that are shared or grow, by sequences alone and among others, with
magnitudes at the types' ends, and with lengths that every key's count shows.

The tolerances of results are those of test_gpu_serving.py; where another is
used, its derivation stands at the test."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from helpers import lib
from test_gpu_serving import _check_prompt, _run_prompt

pytestmark = pytest.mark.gpu

TD = {oracle.F16: torch.float16, oracle.BF16: torch.bfloat16}


@pytest.fixture(scope="module")
def m():
    return lib()


def _randn(seed, *shape, dtype=torch.float16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _filled(m, lens, hk, d, page, seed=0, k=None, v=None, dtype=torch.float16):
    """A cache of sequences of these lengths in shuffled pages, with its table and lengths."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + 1, generator=torch.Generator().manual_seed(seed)).int().cuda()
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    cache, used = m.KVCache.empty(sum(need) + 1, page, hk, d), 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[used:used + need[b]]
        used += need[b]
        at = torch.arange(n, device="cuda")
        cache.write(k[b] if k else _randn(seed + 2 * b + 1, n, hk, d, dtype=dtype), v[b] if v else _randn(seed + 2 * b + 2, n, hk, d, dtype=dtype),
                    table[b, at // page] * page + (at % page).int())
    return cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def _captured(f):
    """f once outside, then in a graph."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f()
    return g


# ------------------------------------------------------------ graphs

def test_graph_of_the_four_operators_replays(m):
    """All four in one graph, replayed on other inputs in the same buffers: bitwise what the calls give."""
    t, hq, hk, d, page = 70, 8, 2, 128, 16
    rope, prompt, decode = m.QKNormRope(hq, hk, d), m.PromptAttention(hq, hk, d), m.CacheAttention(hq, hk, d, page)
    qkv = torch.empty(t, (hq + 2 * hk) * d, dtype=torch.bfloat16, device="cuda")
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hk * d, hk * d], 1))
    qr, kr = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(t, hk, d, dtype=torch.bfloat16, device="cuda")
    out, token = torch.empty_like(qr), torch.empty(1, hq, d, dtype=torch.bfloat16, device="cuda")
    cache, table = m.KVCache.empty(6, page, hk, d), torch.tensor([[4, 1, 5, 0, 2]], dtype=torch.int32, device="cuda")
    at = torch.arange(t, device="cuda")
    slots, cu = table[0, at // page] * page + (at % page).int(), torch.tensor([0, t], dtype=torch.int32, device="cuda")
    n, positions = torch.tensor([t], dtype=torch.int32, device="cuda"), at.int()

    def layer():
        rope.run(q, k, positions, qr, kr)
        cache.write(kr, v, slots)
        prompt.run(qr, kr, v, cu, cu, out)
        decode.run(qr[t - 1:], cache, table, n, token)
    qkv.copy_(_randn(1, t, qkv.shape[1]))
    graph = _captured(layer)
    for seed in (2, 3):
        qkv.copy_(_randn(seed, t, qkv.shape[1]))
        layer()
        want = out.clone(), token.clone()
        out.zero_(), token.zero_(), cache.k.zero_(), cache.v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(token, want[1])
    assert prompt.sync_status() == m.GEMM_OK


def test_graph_keeps_its_workspace_when_the_object_grows(m):
    """The graph's passes cross CTAs, so it goes by the counters in its workspace: what is
    allocated after the growth must not lie there."""
    hq, hk, d, page = 8, 2, 128, 64
    cache, table, n = _filled(m, [20000], hk, d, page)
    op = m.CacheAttention(hq, hk, d, page, dtype=m.GEMM_F16, batch=1)
    q, out = _randn(5, 1, hq, d), torch.empty(1, hq, d, dtype=torch.float16, device="cuda")
    graph = _captured(lambda: op.run(q, cache, table, n, out))
    want, place, size = out.clone(), op.workspace.data_ptr(), op.ws_bytes
    few = torch.tensor([100] * 40, dtype=torch.int32, device="cuda")
    many = torch.empty(40, hq, d, dtype=torch.float16, device="cuda")
    op.run(q.expand(40, hq, d).contiguous(), cache, table.expand(40, -1).contiguous(), few, many)
    assert op.batch >= 40 and op.workspace.data_ptr() != place
    others = [torch.full((size,), 77, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert all(x.data_ptr() >= place + size or x.data_ptr() + size <= place for x in others)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all((x == 77).all() for x in others)


def test_growth_is_refused_while_a_graph_is_captured(m):
    hq, hk, d, page = 4, 2, 64, 16
    cache, table, n = _filled(m, [40, 50, 60], hk, d, page)
    op = m.CacheAttention(hq, hk, d, page, dtype=m.GEMM_F16, batch=1)
    q, out = _randn(6, 3, hq, d), torch.empty(3, hq, d, dtype=torch.float16, device="cuda")
    one = torch.empty(1, hq, d, dtype=torch.float16, device="cuda")
    op.run(q[:1], cache, table[:1], n[:1], one)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    again = torch.empty_like(one)
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="batch=3"):
            op.run(q, cache, table, n, out)
        op.run(q[:1], cache, table[:1], n[:1], again)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, one) and op.batch == 1
    op.run(q, cache, table, n, out)
    assert op.batch == 3 and torch.equal(out[:1], one)


def test_refused_calls_leave_the_workspace(m):
    hq, hk, d, page, n = 4, 2, 64, 16, 90
    cache, table, _ = _filled(m, [40], hk, d, page)
    op = m.CacheAttention(hq, hk, d, page, dtype=m.GEMM_F16, batch=2)
    place = op.workspace.data_ptr()
    ok = dict(q=_randn(7, n, hq, d), cache=cache, page_table=table.expand(n, -1).contiguous(), lengths=torch.full((n,), 40, dtype=torch.int32, device="cuda"),
              out=torch.empty(n, hq, d, dtype=torch.float16, device="cuda"))
    for bad in (dict(q=ok["q"].bfloat16()), dict(q=ok["q"].cpu()), dict(out=ok["out"][:5]), dict(lengths=ok["lengths"].long()),
                dict(page_table=ok["page_table"].t().contiguous().t()), dict(cache=m.KVCache.empty(4, 32, hk, d))):
        with pytest.raises(ValueError):
            op.run(**{**ok, **bad})
        assert op.batch == 2 and op.workspace.data_ptr() == place
    op.run(**ok)
    assert op.batch == n
    with pytest.raises(m.GemmError):  # more than the library takes
        op.run(*(x.expand(8193, *x.shape[1:]).contiguous() if x is not cache else x
                 for x in (ok["q"][:1], cache, table, ok["lengths"][:1], ok["out"][:1])))
    assert op.batch == n


# ------------------------------------------------------------ the cache

def test_cache_pads_with_negative_slots_and_a_doubled_slot_stays_in_its_row(m):
    """A call padded with negative slots writes what the call without them does; what two tokens with one slot
    leave there is unspecified, but every other row of the cache is as if they were not there."""
    hk, d, page, t = 3, 128, 16, 40
    k, v = _randn(10, t, hk, d), _randn(11, t, hk, d, scale=2.0 ** 6)
    k[20:] *= 2.0 ** -7  # (rows of other exponents)
    slots = torch.randperm(4 * page, generator=torch.Generator().manual_seed(0))[:t].int().cuda()
    plain, padded, doubled = (m.KVCache.empty(4, page, hk, d) for _ in range(3))
    for c in (plain, padded, doubled):
        for x in (c.k, c.v, c.k_exp, c.v_exp):
            x.fill_(9)
    plain.write(k[: t - 8], v[: t - 8], slots[: t - 8])
    pad = slots.clone()
    pad[t - 8:] = -1
    padded.write(k, v, pad)
    twice = slots.clone()
    twice[t - 8:] = slots[3]
    doubled.write(k, v, twice)
    for name in ("k", "v", "k_exp", "v_exp"):
        a, b, c = (getattr(x, name).transpose(1, 2).flatten(0, 1) for x in (plain, padded, doubled))  # [slot][head]...
        assert torch.equal(a, b)
        keep = torch.arange(4 * page, device="cuda") != slots[3]
        assert torch.equal(a[keep], c[keep])


# ------------------------------------------------------------ a wait that runs out

def _prompt_case(nq, nk, hq, hk, d, dtype):
    cu_q, cu_k = (torch.tensor([0, *np.cumsum(x)], dtype=torch.int32, device="cuda") for x in (nq, nk))
    return [_randn(20 + i, n, h, d, dtype=TD[dtype]) for i, (n, h) in enumerate(((sum(nq), hq), (sum(nk), hk), (sum(nk), hk)))] + [cu_q, cu_k]


# (the kernels for many units, for few, and for keys cut over clusters of 8 and of 2)
@pytest.mark.parametrize("nq,nk,hq,hk,d,dtype", [
    ([200, 300], [700, 513], 110, 110, 64, oracle.F16), ([500, 520, 9], [500, 520, 700], 128, 32, 128, oracle.BF16),
    ([129, 1, 127, 300], [1290, 1, 700, 300], 2, 2, 128, oracle.F16), ([33, 77], [330, 900], 12, 4, 64, oracle.BF16),
    ([1], [4100], 8, 2, 64, oracle.F16), ([130], [4200], 1, 1, 128, oracle.BF16), ([130], [4200], 30, 30, 64, oracle.BF16)])
def test_prompt_withheld_load_times_out_and_the_next_run_is_right(m, monkeypatch, nq, nk, hq, hk, d, dtype):
    """The waits run out after 20 ms; the status says so once, and the same plan and buffers go on as if nothing had been."""
    args = _prompt_case(nq, nk, hq, hk, d, dtype)
    code = m.GEMM_BF16 if dtype == oracle.BF16 else m.GEMM_F16
    want, out = torch.empty_like(args[0]), torch.empty_like(args[0])
    m.PromptAttention(hq, hk, d, dtype=code).run(*args, want)
    monkeypatch.setenv("LGT_GEMM_WAIT_LIMIT_MS", "20")
    op = m.PromptAttention(hq, hk, d, dtype=code)
    monkeypatch.delenv("LGT_GEMM_WAIT_LIMIT_MS")
    for _ in range(2):
        assert m._lib.attn_prompt_withhold_load(op.plan) == m.GEMM_OK
        op.run(*args, out)
        assert op.sync_status() == m.GEMM_ERR_TIMEOUT and op.sync_status() == m.GEMM_OK
        out.fill_(float("nan"))
        op.run(*args, out)
        assert op.sync_status() == m.GEMM_OK and torch.equal(out, want)


# ------------------------------------------------------------ attention over the cache

def test_one_workspace_serves_any_shape_in_turn(m):
    """Shapes whose parts lie over one another's, each with passes that cross CTAs, so that each goes by the counters."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    runs = []
    for i, (lens, hq, hk, d, dtype) in enumerate([([40000], 8, 2, 64, torch.float16), ([30000, 9000], 8, 1, 128, torch.bfloat16), ([41000], 16, 1, 64, torch.bfloat16),
                                                  ([20000] * 5, 4, 4, 128, torch.float16), ([900] * 70, 24, 8, 64, torch.float16)]):
        cache, table, n = _filled(m, lens, hk, d, 64, seed=100 * i)
        size = ctypes.c_size_t()
        assert m._lib.attn_cache_attend_workspace_size(hq, hk, d, len(lens), ctypes.byref(size)) == m.GEMM_OK
        assert sum(-(-x // 16) for x in lens) * hk > 16 * sms  # more than a block of keys for every warp
        runs.append((cache, table, n, _randn(200 + i, len(lens), hq, d, dtype=dtype), hq, m.GEMM_BF16 if dtype is torch.bfloat16 else m.GEMM_F16, size.value))
    shared = torch.zeros(max(r[-1] for r in runs), dtype=torch.uint8, device="cuda")

    def run(r, workspace):
        cache, table, n, q, hq, code, size = r
        out = torch.full_like(q, float("nan"))
        st = m._lib.attn_cache_attend(cache._ref, q.data_ptr(), 0, hq, table.data_ptr(), 0, table.shape[1], n.data_ptr(), len(q), 0.0, code, out.data_ptr(), 0,
                                      workspace.data_ptr(), workspace.numel(), torch.cuda.current_stream().cuda_stream)
        assert st == m.GEMM_OK
        return out
    want = [run(r, torch.zeros(r[-1], dtype=torch.uint8, device="cuda")) for r in runs]
    assert all(torch.isfinite(x).all() for x in want)
    for i in [0, 1, 0, 2, 1, 3, 0, 4, 2, 4, 3, 1, 0, 0]:
        assert torch.equal(run(runs[i], shared), want[i]), i


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [-126, -20, 120, 126, 127])
def test_decode_queries_of_any_size(m, d, power):
    """bf16 queries up to the type's largest and down to its subnormals, over keys and with a scale that bring the
    logits back to where they were.  Queries are multiples of 2^-6 below 2, so every form of them is exact and
    all else differs by powers of two: the results are bitwise those of the queries as they were."""
    hq, hk, n, page = 4, 2, 300, 16
    q = _randn(30, 1, hq, d, dtype=torch.float64)
    q = ((q * (127 / q.abs().amax(-1, keepdim=True))).round() / 64).bfloat16()  # the largest of a head in [1, 2)
    near = m.KVCache.empty(20, page, hk, d)
    slots, table = torch.arange(n, dtype=torch.int32, device="cuda"), torch.arange(20, dtype=torch.int32, device="cuda")[None]
    lengths, scale = torch.tensor([n], dtype=torch.int32, device="cuda"), float(np.float32(1 / np.sqrt(d)))
    want, got = torch.empty_like(q), torch.empty_like(q)
    near.write(_randn(31, n, hk, d, dtype=torch.bfloat16, scale=2.0), _randn(32, n, hk, d, dtype=torch.bfloat16), slots)
    m.CacheAttention(hq, hk, d, page, scale=scale).run(q, near, table, lengths, want)
    # queries times 2^power, keys over 2^shift, the rest in the scale
    shift = max(min(power, 100), -100)
    far = m.KVCache(near.k, near.v, (near.k_exp.int() - shift).to(torch.uint8), near.v_exp)
    big = (q.double() * 2.0 ** power).bfloat16()
    assert torch.equal(big.double() * 2.0 ** -power, q.double())
    m.CacheAttention(hq, hk, d, page, scale=scale * 2.0 ** (shift - power)).run(big, far, table, lengths, got)
    assert torch.equal(got, want) and want.abs().max() > 0.1


@pytest.mark.parametrize("d", [64, 128])
def test_decode_very_large_keys_under_very_small_queries(m, d):
    """Logits of size 10 from keys near the type's largest and queries near its smallest, as above bitwise those of
    keys and queries near 1; and logits of 0 from keys and queries that are both very large."""
    hq, hk, n, page = 4, 2, 300, 16
    q = _randn(33, 1, hq, d, dtype=torch.float64)
    q = ((q * (127 / q.abs().amax(-1, keepdim=True))).round() / 64).bfloat16()
    near = m.KVCache.empty(20, page, hk, d)
    slots, table = torch.arange(n, dtype=torch.int32, device="cuda"), torch.arange(20, dtype=torch.int32, device="cuda")[None]
    lengths, want, got = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.empty_like(q), torch.empty_like(q)
    near.write(_randn(34, n, hk, d, dtype=torch.bfloat16, scale=0.5), _randn(35, n, hk, d, dtype=torch.bfloat16), slots)
    op = m.CacheAttention(hq, hk, d, page, scale=1.0)
    op.run(q, near, table, lengths, want)
    op.run((q.double() * 2.0 ** -126).bfloat16(), m.KVCache(near.k, near.v, (near.k_exp.int() + 126).to(torch.uint8), near.v_exp), table, lengths, got)
    assert torch.isfinite(want).all() and torch.equal(got, want)
    k = torch.zeros(n, hk, d, dtype=torch.bfloat16, device="cuda")
    k[:, :, 1::2] = 2.0 ** 120
    q = torch.zeros_like(q)
    q[:, :, ::2] = 2.0 ** 100
    v = torch.ones_like(k)
    v[:, :, 0] = torch.arange(n, device="cuda")[:, None] % 2
    near.write(k, v, slots)
    op.run(q, near, table, lengths, got)
    # (half the keys have the value 1: weights and sums are exact, the one rounding is that of 1 over the sum)
    assert torch.all(got[:, :, 1:] == 1) and torch.all(got[:, :, 0] == 0.5)


@pytest.mark.parametrize("hq,hk,d", [(8, 1, 128), (6, 2, 64)])
def test_decode_sequences_alone_and_among_others(m, hq, hk, d):
    """The rest of the batch decides where a sequence's keys are cut, and each cut rounds the weights anew: 2^-11 S
    either side, with S <= max |v|, the results' own roundings 2^-11 |r| either side, n 2^-24 max |v| of fp32 and
    subnormal weights.  A sequence of one block of keys is not cut, and in the same batch nothing changes."""
    lens, page = [2000, 1, 900, 3500, 16, 5000, 311, 1800], 16
    k, v = ([_randn(40 + 2 * b + i, n, hk, d) for b, n in enumerate(lens)] for i in range(2))
    cache, table, n = _filled(m, lens, hk, d, page, k=k, v=v)
    q = _randn(60, len(lens), hq, d, scale=3.0)
    op, out, again, alone = m.CacheAttention(hq, hk, d, page, dtype=m.GEMM_F16), torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    op.run(q, cache, table, n, out)
    op.run(q, cache, table, n, again)
    assert torch.equal(out, again)
    for b in range(len(lens)):
        op.run(q[b:b + 1], cache, table[b:b + 1], n[b:b + 1], alone[b:b + 1])
        most = float(v[b].abs().max()) * 1.0625  # (as e4m3 holds it)
        tol = 2.0 ** -10 * out[b].float().abs() + (2.0 ** -10 + lens[b] * 2.0 ** -24) * most
        assert torch.all((alone[b].float() - out[b].float()).abs() <= tol), lens[b]
        assert lens[b] > page or torch.equal(alone[b], out[b])


# ------------------------------------------------------------ packed attention: many sequences

def _spread(batch, tokens, seed):
    """`tokens` tokens in runs of 1 to 3 over `batch` sequences, most of which may be empty; the last has some."""
    rng = np.random.default_rng(seed)
    n = np.zeros(batch, dtype=np.int64)
    for b in [batch - 1, *rng.permutation(batch - 1)]:
        n[b] = min(int(rng.integers(1, 4)), tokens - n.sum())
    return n


# (the kernels for many units, for few, and for keys cut over clusters)
@pytest.mark.parametrize("batch,tokens,keys,hq,hk,d,dtype", [(3000, 5000, 1, 4, 2, 64, oracle.F16), (700, 1200, 9, 6, 3, 128, oracle.BF16),
                                                             (3000, 40, 30, 4, 2, 128, oracle.F16), (2000, 2, 4500, 4, 1, 64, oracle.BF16)])
def test_prompt_many_sequences(m, batch, tokens, keys, hq, hk, d, dtype):
    """Far more sequences than a warp looks at a time, runs of empty ones among them."""
    nq = _spread(batch, tokens, batch)
    nk = nq * keys
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (nq, nk))
    q, k, v = (_randn(70 + i, int(n), h, d, dtype=TD[dtype]).cpu() for i, (n, h) in enumerate(((nq.sum(), hq), (nk.sum(), hk), (nk.sum(), hk))))
    got = _run_prompt(m, q, k, v, cu_q, cu_k, dtype)
    _check_prompt(got, q, k, v, cu_q, cu_k, dtype, what=str((batch, tokens)))
    assert torch.equal(got, _run_prompt(m, q, k, v, cu_q, cu_k, dtype))


def test_prompt_sequences_are_limited(m):
    x, cu = _randn(75, 8, 2, 64), torch.zeros((1 << 20) + 2, dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 3.0)
    op = m.PromptAttention(2, 2, 64, dtype=m.GEMM_F16)
    with pytest.raises(m.GemmError):
        op.run(x, x, x, cu, cu, out)
    cu[-2:] = 8
    op.run(x, x, x, cu[:-1], cu[:-1], out)  # 2^20: all tokens are the last sequence's
    want = torch.empty_like(x)
    few = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    op.run(x, x, x, few, few, want)
    assert op.sync_status() == m.GEMM_OK and torch.equal(out, want)


# ------------------------------------------------------------ every key counts once

def _marked_values(n, hk, d, dtype):
    """Values [n][hk][d] that are 1 in one column, another for each run of n / d keys, and 0 elsewhere; and the keys of
    a run.  Under queries of 0 every visible key has the same weight, exactly, so a result's column is the number of
    visible keys of its run over that of all: a key left out, or taken twice, of a run of 512 changes it by 2^-9."""
    run = -(-n // d)
    v = torch.zeros(n, hk, d, dtype=dtype, device="cuda")
    at = torch.arange(n, device="cuda")
    v[at, :, at // run] = 1.0
    return v, run


def _shares(seen, run, d):
    """What the columns are for rows that see this many keys."""
    seen = seen.double()[:, None]
    return (seen - run * torch.arange(d, device="cuda")).clamp(0, run) / seen


@pytest.mark.parametrize("lens,hq,hk,d", [
    ([65536], 16, 1, 128), ([65536], 1, 1, 128), ([60000], 8, 1, 64), ([30000, 7, 20000], 8, 4, 128), ([1000] * 40, 12, 2, 64),
    ([17 * i + 1 for i in range(200)], 4, 2, 128), ([100] * 300, 2, 1, 64)])
def test_decode_counts_every_key_once(m, lens, hq, hk, d):
    """Passes over 1 to 152 CTAs, joined in groups of 32.  Weights and sums are exact, so a result is off by its one
    rounding and that of the quotient in fp32."""
    page = 16
    marked = [_marked_values(n, hk, d, torch.float16) for n in lens]
    cache, table, n = _filled(m, lens, hk, d, page, v=[x for x, _ in marked])
    q = torch.zeros(len(lens), hq, d, dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    m.CacheAttention(hq, hk, d, page, dtype=m.GEMM_F16).run(q, cache, table, n, out)
    for b, length in enumerate(lens):
        want = _shares(n[b:b + 1], marked[b][1], d)
        assert torch.all((out[b].double() - want).abs() <= (2.0 ** -11 + 2.0 ** -20) * want + 2.0 ** -25), (b, length)


# (keys cut over clusters of 8, 8, 4 and 2; the kernel for few units, and for many)
@pytest.mark.parametrize("nq,nk,hq,hk,d,dtype", [
    ([3], [150000], 1, 1, 64, oracle.BF16), ([1, 20], [32768, 9000], 8, 2, 128, oracle.F16), ([64], [20000], 24, 6, 128, oracle.F16),
    ([130], [6000], 30, 30, 64, oracle.F16), ([300, 40], [20000, 700], 40, 40, 64, oracle.F16), ([300, 500], [5000, 300], 110, 110, 64, oracle.F16),
    ([700, 1, 90], [3000, 4000, 90], 128, 32, 128, oracle.F16)])
def test_prompt_counts_every_key_once(m, nq, nk, hq, hk, d, dtype):
    """As for the cache: weights of 1 and sums below 2^24 are exact in either type."""
    op = m.PromptAttention(hq, hk, d, dtype=m.GEMM_BF16 if dtype == oracle.BF16 else m.GEMM_F16)
    marked = [_marked_values(n, hk, d, TD[dtype]) for n in nk]
    v = torch.cat([x for x, _ in marked])
    k, q = _randn(80, *v.shape, dtype=TD[dtype]), torch.zeros(sum(nq), hq, d, dtype=TD[dtype], device="cuda")
    cu_q, cu_k = (torch.tensor([0, *np.cumsum(x)], dtype=torch.int32, device="cuda") for x in (nq, nk))
    out = torch.empty_like(q)
    op.run(q, k, v, cu_q, cu_k, out)
    assert op.sync_status() == m.GEMM_OK
    u = 2.0 ** (-8 if dtype == oracle.BF16 else -11)
    for b, (a, n) in enumerate(zip(nq, nk)):
        seen = (torch.arange(a, device="cuda") + n - a + 1).clamp(0, n)
        rows = out[int(cu_q[b]):int(cu_q[b + 1])].double()
        want = torch.where(seen[:, None] > 0, _shares(seen.clamp(min=1), marked[b][1], d), 0.0)[:, None]
        assert torch.all((rows - want).abs() <= (u + 2.0 ** -20) * want + 2.0 ** -25), b


# ------------------------------------------------------------ the size of errors over long keys

def _rms_of_rounded_weights(weights, v, out, u_w, u):
    """The rms error of sums of rounded weights times values [n][d], themselves rounded: a rounding is off by u / sqrt 3
    of its value in the mean square, and roundings are independent.  (At most u, so where one weight is all of a
    result, sqrt 3 of it.)"""
    return float(((u_w ** 2 * (weights ** 2 @ v ** 2) + u ** 2 * out ** 2) / 3).mean().sqrt())


@pytest.mark.parametrize("scale", [0.125, 1.0])
def test_prompt_error_over_long_keys_is_that_of_rounded_weights(m, scale):
    """bf16 weights have fp32's range, so nothing is lost however many keys there are: rms within twice the roundings'."""
    nq, n, d = 3, 150000, 64
    q, k, v = (_randn(90 + i, x, 1, d, dtype=torch.bfloat16) for i, x in enumerate((nq, n, n)))
    cu_q, cu_k, out = torch.tensor([0, nq], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.empty_like(q)
    m.PromptAttention(1, 1, d, scale=scale).run(q, k, v, cu_q, cu_k, out)
    logits = q[:, 0].double() @ k[:, 0].double().T * scale
    logits.masked_fill_(torch.triu(torch.ones(nq, n, dtype=torch.bool, device="cuda"), n - nq + 1), -float("inf"))
    weights = torch.softmax(logits, -1)
    want = weights @ v[:, 0].double()
    rms = float((out[:, 0].double() - want).square().mean().sqrt())
    assert rms <= 2 * _rms_of_rounded_weights(weights, v[:, 0].double(), want, 2.0 ** -8, 2.0 ** -8)


@pytest.mark.parametrize("n,hq,hk,d,dtype", [(20000, 8, 8, 64, oracle.F16), (60000, 8, 1, 128, oracle.F16), (60000, 2, 1, 128, oracle.BF16)])
def test_decode_error_over_long_keys_is_that_of_rounded_weights(m, n, hq, hk, d, dtype):
    """fp16 weights, the largest contribution's in its middle: those of logits of size 1 all lie above 2^-14 of it."""
    page = 64
    cache, table, lengths = _filled(m, [n], hk, d, page, seed=7, dtype=TD[dtype])
    q, out = _randn(95, 1, hq, d, dtype=TD[dtype]), torch.empty(1, hq, d, dtype=TD[dtype], device="cuda")
    m.CacheAttention(hq, hk, d, page, dtype=m.GEMM_BF16 if dtype == oracle.BF16 else m.GEMM_F16).run(q, cache, table, lengths, out)
    at = torch.arange(n, device="cuda")
    slots = table[0, at // page] * page + (at % page).int()
    k, v = (torch.empty(n, hk, d, dtype=TD[dtype], device="cuda") for _ in range(2))
    cache.read(slots, k, v)  # (exact: the codes' values of rows of this size are values of either type)
    for h in range(hq):
        kv = h // (hq // hk)
        weights = torch.softmax(q[:, h].double() @ k[:, kv].double().T / d ** 0.5, -1)
        want = weights @ v[:, kv].double()
        rms = float((out[:, h].double() - want).square().mean().sqrt())
        assert rms <= 2 * _rms_of_rounded_weights(weights, v[:, kv].double(), want, 2.0 ** -11, 2.0 ** (-8 if dtype == oracle.BF16 else -11)), h
