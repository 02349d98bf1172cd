"""CPU tests of the serving operators' host side: the refusals of every entry
point, the rotation's frequencies, the oracle's own pins, and the split of the
cache attention's work, restated here from its integer formulas.  No GPU work."""
import ctypes

import numpy as np
import pytest

import oracle


@pytest.fixture(scope="module")
def lib():
    import helpers
    return helpers.lib()


def _rope_desc(lib, **kw):
    a = dict(q_heads=4, k_heads=2, head_dim=64, rot_dim=64, layout=lib.ATTN_ROPE_HALF, dtype=lib.GEMM_BF16, eps=1e-6,
             magnitude=1.0, base=10000.0, factor=1.0, context=0.0, low_turns=0.0, high_turns=0.0)
    a.update(kw)
    return lib.attn_rope_desc_t(*a.values())


@pytest.mark.parametrize("kw", [dict(rot=128, base=10000.0), dict(rot=64, base=500000.0, factor=8.0, context=8192.0, low=1.0, high=4.0),
                                dict(rot=32, base=10000.0, factor=4.0), dict(rot=16, base=100.0, factor=2.0, context=50.0, low=3.0, high=3.0)])
def test_rope_frequencies(lib, kw):
    d = _rope_desc(lib, head_dim=128, rot_dim=kw["rot"], base=kw["base"], factor=kw.get("factor", 1.0),
                   context=kw.get("context", 0.0), low_turns=kw.get("low", 0.0), high_turns=kw.get("high", 0.0))
    want = oracle.rope_frequencies(**kw)
    assert np.allclose(lib.attn_rope_frequencies(d), want, rtol=1e-14, atol=0)
    if kw.get("factor", 1.0) > 1 and not kw.get("high"):
        assert np.allclose(want, oracle.rope_frequencies(kw["rot"], kw["base"]) / kw["factor"], rtol=1e-15)


@pytest.mark.parametrize("kw", [dict(q_heads=0), dict(k_heads=0), dict(head_dim=0), dict(head_dim=60), dict(head_dim=264),
                                dict(rot_dim=-8), dict(rot_dim=72), dict(rot_dim=12), dict(layout=2), dict(dtype=3),
                                dict(eps=-1.0), dict(eps=float("nan")), dict(magnitude=float("inf")), dict(base=0.0),
                                dict(base=float("nan")), dict(factor=0.5), dict(factor=float("inf")),
                                dict(low_turns=2.0, high_turns=1.0), dict(low_turns=-1.0),
                                dict(factor=2.0, low_turns=1.0, high_turns=4.0)])
def test_rope_refuses_descriptions(lib, kw):
    st, h = lib.attn_rope_create_status(_rope_desc(lib, **kw))
    assert st == lib.GEMM_ERR_INVALID_ARG and not h


def test_rope_refuses_frequencies_and_pointers(lib):
    d = _rope_desc(lib)
    assert lib.attn_rope_create_status(d, [float("nan")] * 32)[0] == lib.GEMM_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        lib.QKNormRope(4, 2, 64, frequencies=[1.0] * 31)
    st, h = lib.attn_rope_create_status(d, [0.1] * 32)
    assert st == lib.GEMM_OK and h
    run = lib._lib.attn_rope_run
    ok = dict(Q=1 << 20, qs=0, K=1 << 21, ks=0, wq=None, wk=None, pos=1 << 22, n=5, qo=1 << 23, qos=0, ko=1 << 24, kos=0)

    def status(**kw):
        return run(h, *{**ok, **kw}.values(), None)
    assert status(n=-1) == lib.GEMM_ERR_INVALID_ARG
    for name in ("Q", "K", "pos", "qo", "ko"):
        assert status(**{name: None}) == lib.GEMM_ERR_INVALID_ARG
    for name, bad in (("qs", 255), ("qs", 260), ("ks", 120), ("qos", 248), ("kos", 129)):
        assert status(**{name: bad}) == lib.GEMM_ERR_INVALID_ARG
    for name in ("Q", "K", "qo", "ko"):
        assert status(**{name: ok[name] + 8}) == lib.GEMM_ERR_ALIGNMENT
    assert status(wq=8) == lib.GEMM_ERR_ALIGNMENT and status(pos=(1 << 22) + 2) == lib.GEMM_ERR_ALIGNMENT
    assert status(n=1 << 40) == lib.GEMM_ERR_UNSUPPORTED
    assert status(n=0, Q=None, K=None, pos=None, qo=None, ko=None) == lib.GEMM_OK
    assert run(None, *ok.values(), None) == lib.GEMM_ERR_INVALID_ARG
    assert lib._lib.attn_rope_destroy(h) == lib.GEMM_OK and lib._lib.attn_rope_destroy(None) == lib.GEMM_OK


@pytest.mark.parametrize("kw", [dict(q_heads=0), dict(k_heads=0), dict(q_heads=5), dict(q_heads=258), dict(head_dim=96),
                                dict(dtype=2), dict(causal=2), dict(scale=-1.0), dict(scale=float("nan")),
                                dict(scale=float("inf"))])
def test_prompt_refuses_descriptions(lib, kw):
    a = dict(q_heads=4, k_heads=2, head_dim=64, dtype=lib.GEMM_F16, causal=1, scale=0.0)
    a.update(kw)
    st, h = lib.attn_prompt_create_status(lib.attn_prompt_desc_t(*a.values()))
    assert st == lib.GEMM_ERR_INVALID_ARG and not h


def test_cache_entry_points_refuse(lib):
    def cache(**kw):
        a = dict(k=1 << 20, v=1 << 24, k_exp=1 << 28, v_exp=1 << 29, pages=4, page_size=32, k_heads=2, head_dim=64)
        a.update(kw)
        return ctypes.byref(lib.attn_cache_t(*a.values()))
    ok = dict(K=1 << 30, ks=0, V=1 << 31, vs=0, slots=1 << 32, n=3, dtype=lib.GEMM_F16)

    def write(c, **kw):
        return lib._lib.attn_cache_write(c, *{**ok, **kw}.values(), None)

    def read(c, **kw):
        a = {**ok, **kw}
        return lib._lib.attn_cache_read(c, a["slots"], a["n"], a["K"], a["ks"], a["V"], a["vs"], a["dtype"], None)
    for f in (write, read):
        for kw in (dict(k=None), dict(v=None), dict(k_exp=None), dict(v_exp=None), dict(pages=0), dict(pages=1 << 31),
                   dict(page_size=8), dict(page_size=40), dict(page_size=2048), dict(k_heads=0), dict(head_dim=96)):
            assert f(cache(**kw)) == lib.GEMM_ERR_INVALID_ARG, kw
        assert f(None) == lib.GEMM_ERR_INVALID_ARG
        for kw in (dict(K=None), dict(V=None), dict(slots=None), dict(ks=120), dict(vs=132), dict(n=-1), dict(dtype=2)):
            assert f(cache(), **kw) == lib.GEMM_ERR_INVALID_ARG, kw
        for kw in (dict(K=(1 << 30) + 8), dict(V=(1 << 31) + 2), dict(slots=(1 << 32) + 1)):
            assert f(cache(), **kw) == lib.GEMM_ERR_ALIGNMENT, kw
        assert f(cache(k=(1 << 20) + 8)) == lib.GEMM_ERR_ALIGNMENT
        assert f(cache(), n=1 << 31) == lib.GEMM_ERR_UNSUPPORTED
        assert f(cache(), n=0, K=None, V=None, slots=None) == lib.GEMM_OK

    a = dict(Q=1 << 30, qs=0, hq=4, table=1 << 31, ts=0, pages=9, lengths=1 << 32, batch=3, scale=0.0, dtype=lib.GEMM_F16,
             out=1 << 33, os=0, ws=1 << 34, wsb=1 << 40)

    def attend(c, **kw):
        return lib._lib.attn_cache_attend(c, *{**a, **kw}.values(), None)
    for kw in (dict(Q=None), dict(out=None), dict(table=None), dict(lengths=None), dict(hq=3), dict(hq=0), dict(batch=-1),
               dict(scale=-1.0), dict(scale=float("nan")), dict(qs=248), dict(os=260), dict(ts=8), dict(pages=-1), dict(dtype=1 << 8)):
        assert attend(cache(), **kw) == lib.GEMM_ERR_INVALID_ARG, kw
    for kw in (dict(Q=(1 << 30) + 8), dict(out=(1 << 33) + 2), dict(table=(1 << 31) + 2), dict(lengths=(1 << 32) + 1)):
        assert attend(cache(), **kw) == lib.GEMM_ERR_ALIGNMENT, kw
    assert attend(cache(), batch=8193) == lib.GEMM_ERR_UNSUPPORTED
    assert attend(cache(), pages=1 << 26) == lib.GEMM_ERR_UNSUPPORTED
    assert attend(cache(), batch=0, Q=None, out=None) == lib.GEMM_OK
    n = ctypes.c_size_t()
    size = lib._lib.attn_cache_attend_workspace_size
    assert size(4, 3, 64, 1, ctypes.byref(n)) == lib.GEMM_ERR_INVALID_ARG
    assert size(4, 2, 64, 1, None) == lib.GEMM_ERR_INVALID_ARG
    assert size(4, 2, 64, 8193, ctypes.byref(n)) == lib.GEMM_ERR_UNSUPPORTED


def test_host_tensors_are_refused(lib):
    import torch
    x, i = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(4, dtype=torch.int32)
    k = torch.zeros(3, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        lib.QKNormRope(4, 2, 64, dtype=lib.GEMM_F16).run(x, k, i[:3], x, k)
    with pytest.raises(ValueError):
        lib.KVCache(*[torch.zeros(2, 2, 16, 64, dtype=torch.uint8)] * 2, *[torch.zeros(2, 2, 16, dtype=torch.uint8)] * 2)


def test_oracle_codes():
    """Pins: the extremes of the code table, ties, the choice of the power and what is not finite."""
    grid = oracle._e4m3_values()
    assert grid[0] == 0 and grid[1] == 2.0 ** -9 and grid[8] == 2.0 ** -6 and grid[126] == 448.0 and len(set(grid)) == 127
    import torch
    x = torch.randn(4000, dtype=torch.float64).mul(60).clamp(-448, 448).float()
    codes, exps = oracle.cache_encode(np.concatenate([x.numpy().astype(np.float64), [448.0]])[None])
    assert exps[0] == 127
    assert np.array_equal(codes[0, :-1], x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    for amax, power in ((448.0, 0), (449.0, 1), (224.0, -1), (1.75, -8), (1.7500001, -7), (2.0 ** -133, -126), (0.0, 0)):
        assert oracle.cache_encode(np.array([[amax, 0.0]]))[1][0] == power + 127
    codes, exps = oracle.cache_encode(np.array([[np.inf, -np.inf, np.nan, 1.0]]))
    assert list(codes[0]) == [126, 254, 127, 0x78] and exps[0] == 127 - 8
    assert np.array_equal(oracle.cache_decode(*oracle.cache_encode(np.array([[3.0, -0.25, 448 * 2.0]]))), [[3.0, -0.25, 896.0]])


def test_oracle_attention_is_the_dense_one():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(5, 2, 8)), rng.normal(size=(9, 1, 8)), rng.normal(size=(9, 1, 8))
    out, mag = oracle.prompt_attention(q, k, v, [0, 5], [0, 9], causal=False)
    for h in range(2):
        assert np.allclose(out[:, h], oracle._softmax_rows(q[:, h] @ k[:, 0].T / np.sqrt(8)) @ v[:, 0])
    out, _ = oracle.prompt_attention(q, k, v, [0, 5], [0, 3], causal=True)
    assert not out[:2].any() and np.allclose(out[2, 0], v[0, 0])


def test_cache_attention_split_covers_every_unit_once():
    """The CTAs' runs of units partition them and none is empty, the warps'
    runs partition a CTA's, and the CTAs that take part in a range of units
    are exactly those between the owners of its first and last."""
    rng = np.random.default_rng(1)
    for _ in range(300):
        total, grid, warps = int(rng.integers(1, 5000)), int(rng.integers(1, 400)), int(rng.choice([8, 16]))
        ctas = min(grid, max(total // warps, 1))
        start = [c * total // ctas for c in range(ctas + 1)]
        assert start[0] == 0 and start[-1] == total and all(a < b for a, b in zip(start, start[1:]))
        for t0, t1 in zip(start, start[1:]):
            runs = [t0 + (t1 - t0) * w // warps for w in range(warps + 1)]
            assert runs[0] == t0 and runs[-1] == t1 and (total < warps or all(a < b for a, b in zip(runs, runs[1:])))
        owner = [((t + 1) * ctas - 1) // total for t in range(total)]
        for t in range(total):
            assert start[owner[t]] <= t < start[owner[t] + 1]
        a = int(rng.integers(0, total))
        b = int(rng.integers(a, total))
        part = {c for c in range(ctas) if start[c] <= b and start[c + 1] > a}
        assert part == set(range(owner[a], owner[b] + 1))
