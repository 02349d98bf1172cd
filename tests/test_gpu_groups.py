"""Rows in groups on the GPU: row_groups, GroupedGemm and GroupedGemmK against
their definitions in 64 bits.

Most inputs are small whole numbers, so every sum is below 2^24 and exact in
fp32: the result is then the exact sum rounded once to the output type, and has
to be equal to it, bit by bit.  For normal inputs the tolerance is half a step of
the output type (torch.finfo(t).eps / 2 of the value) and, for the sums, two
roundings of 2^-24 at a magnitude of at most sum |a b| / sqrt(K) * 8 for each of
the K terms, in the mean of K signs: sqrt(K) * 2 * 2^-24 * 8 / sqrt(K) * sum |a b|
= 2^-20 sum |a b|."""
import random

import numpy as np
import pytest
import torch

from helpers import lib

pytestmark = pytest.mark.gpu

TD = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def m():
    return lib()


def _code(m, t):
    return m.GEMM_BF16 if t == "bf16" else m.GEMM_F16


def _ints(seed, *shape, dtype, most=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(dtype)


def _pitched(t, extra):
    """t with rows `extra` values longer, which hold NaN."""
    if not extra:
        return t
    wide = torch.full((*t.shape[:-1], t.shape[-1] + extra), float("nan"), dtype=t.dtype, device="cuda")
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


def _offsets(sizes, start=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]) + start, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ row_groups

def _check_groups(m, ids, groups, places=True):
    n = len(ids)
    offsets = torch.full((groups + 1,), -7, dtype=torch.int32, device="cuda")
    order = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    back = torch.full((n,), -7, dtype=torch.int32, device="cuda") if places else None
    m.row_groups(ids, offsets, order, back)
    host = ids.cpu().numpy().astype(np.int64)
    key = np.where((host < 0) | (host >= groups), groups, host)
    want = np.argsort(key, kind="stable")
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(key, minlength=groups + 1)[:groups])]))
    assert np.array_equal(order.cpu().numpy(), want)
    if places:
        assert np.array_equal(back.cpu().numpy(), np.argsort(want, kind="stable"))


@pytest.mark.parametrize("rows", [0, 1, 31, 32, 33, 1000, 1024, 4096, 4097, 8191, 40000, 131072, 300001])
@pytest.mark.parametrize("groups", [1, 5, 128, 1024])
def test_row_groups(m, rows, groups):
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + groups)
    ids = torch.randint(-2, groups + 2, (rows,), generator=g, device="cuda", dtype=torch.int32)
    _check_groups(m, ids, groups, places=rows % 2 == 1)


@pytest.mark.parametrize("kind", ["one", "none", "last", "steps", "far"])
def test_row_groups_lopsided(m, kind):
    n, groups = 20011, 77
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    if kind == "none":
        ids -= 1
    elif kind == "last":
        ids += groups - 1
    elif kind == "steps":
        ids = (torch.arange(n, device="cuda") // 300).int()
    elif kind == "far":
        ids = torch.tensor([-2**31, 2**31 - 1, groups, -1, 0] * (n // 5), dtype=torch.int32, device="cuda")
    _check_groups(m, ids, groups)


# ------------------------------------------------------------------ groups along M

def _rows_reference(a, b, at, k_contig):
    out = {}
    for g in range(len(at) - 1):
        lo, hi = at[g], at[g + 1]
        if hi > lo:
            w = b[g].double()
            out[(lo, hi)] = a[lo:hi].double() @ (w.T if k_contig else w)
    return out


def _check_rows(m, sizes, n, k, k_contig, dtype, pad=0, start=0, extra=(0, 0, 0), seed=0):
    t, rows = TD[dtype], sum(sizes) + pad + start
    a = _pitched(_ints(seed, rows, k, dtype=t), extra[0])
    b = _pitched(_ints(seed + 1, len(sizes), *((n, k) if k_contig else (k, n)), dtype=t), extra[1])
    c = _pitched(torch.full((rows, n), -77.0, dtype=t, device="cuda"), extra[2])
    offsets = _offsets(sizes, start)
    if start:
        a[:start] = float("nan")
    if pad:
        a[rows - pad:] = float("inf")
    op = m.GroupedGemm(len(sizes), n, k, b_layout=m.GEMM_K_CONTIG if k_contig else m.GEMM_MN_CONTIG, dtype=_code(m, dtype))
    op.run(a, b, offsets, c)
    assert op.sync_status() == m.GEMM_OK
    want = torch.full((rows, n), -77.0, dtype=t, device="cuda")
    for (lo, hi), v in _rows_reference(a, b, offsets.tolist(), k_contig).items():
        want[lo:hi] = v.to(t)
    assert torch.equal(c, want), (c != want).nonzero()[:5]
    op.close()


SIZES = [[1], [0, 1, 0], [16], [17, 0, 3], [5] * 40, [0] * 9 + [31], [33, 1, 128, 64], [130, 250, 1, 0, 257, 90], [600, 513],
         [97] * 7, [1000, 0, 0, 3, 24], [256, 512, 255], [1] * 200]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}_{sum(s)}")
@pytest.mark.parametrize("k_contig", [True, False])
@pytest.mark.parametrize("n,k", [(8, 8), (136, 72), (264, 200), (512, 1000)])
def test_rows(m, sizes, k_contig, n, k):
    _check_rows(m, sizes, n, k, k_contig, "bf16" if (n + len(sizes)) % 16 else "f16", seed=len(sizes))


@pytest.mark.parametrize("k_contig", [True, False])
@pytest.mark.parametrize("sizes", [[3, 0, 20], [200, 111, 300]], ids=["few", "many"])
def test_rows_strided_padded(m, sizes, k_contig):
    _check_rows(m, sizes, 264, 136, k_contig, "f16", pad=19, start=5, extra=(8, 16, 24), seed=3)
    _check_rows(m, sizes, 264, 136, k_contig, "bf16", pad=300, start=130, extra=(0, 8, 0), seed=4)


@pytest.mark.parametrize("groups", [255, 256, 257, 1024])
def test_rows_many_groups(m, groups):
    r = random.Random(groups)
    _check_rows(m, [r.choice((0, 0, 1, 2, 40)) for _ in range(groups)], 72, 64, groups % 2 == 0, "bf16", seed=groups)
    _check_rows(m, [r.choice((0, 100, 300)) for _ in range(groups)], 136, 64, groups % 2 == 0, "f16", seed=groups)


@pytest.mark.parametrize("sizes", [[1], [0, 5, 0, 16], [40], [200], [3, 60, 1, 17, 130, 9], [0, 0]], ids=lambda s: f"{len(s)}x{max(s)}_{sum(s)}")
@pytest.mark.parametrize("k_contig", [True, False])
@pytest.mark.parametrize("n,k", [(8, 1304), (136, 712), (200, 4096), (1024, 2000)])
def test_rows_few_tiles(m, sizes, k_contig, n, k):
    """Tiles too few for the SMs: K is split over clusters of two to eight CTAs."""
    _check_rows(m, sizes, n, k, k_contig, "bf16" if (n + len(sizes)) % 16 else "f16", pad=3, start=2, extra=(8, 0, 8), seed=len(sizes))


# ------------------------------------------------------------------ groups along K

def _check_sums(m, sizes, mm, n, dtype, pad=0, start=0, extra=(0, 0, 0), seed=0):
    t, rows = TD[dtype], sum(sizes) + pad + start
    a, b = _pitched(_ints(seed, rows, mm, dtype=t), extra[0]), _pitched(_ints(seed + 1, rows, n, dtype=t), extra[1])
    c = _pitched(torch.full((len(sizes), mm, n), -77.0, dtype=t, device="cuda"), extra[2])
    offsets = _offsets(sizes, start)
    for x in (a, b):
        x[:start] = float("nan")
        x[rows - pad:] = float("inf")
    op = m.GroupedGemmK(len(sizes), mm, n, dtype=_code(m, dtype))
    op.run(a, b, offsets, c)
    assert op.sync_status() == m.GEMM_OK
    at = offsets.tolist()
    for g in range(len(sizes)):
        want = (a[at[g]:at[g + 1]].double().T @ b[at[g]:at[g + 1]].double()).to(t)
        assert torch.equal(c[g], want), (g, (c[g] != want).nonzero()[:5])
    op.close()


SUM_SIZES = [[0], [1], [0, 0, 7, 0], [64], [65, 63], [128, 1, 0, 15, 16, 17], [5] * 40, [31, 33, 47, 48, 49, 63, 64, 65, 80], [1000, 24], [700, 0, 901]]


@pytest.mark.parametrize("sizes", SUM_SIZES, ids=lambda s: f"{len(s)}x{max(s)}_{sum(s)}")
@pytest.mark.parametrize("mm,n", [(8, 8), (64, 520), (72, 136), (264, 200), (1000, 512), (520, 120)])
def test_sums(m, sizes, mm, n):
    _check_sums(m, sizes, mm, n, "bf16" if (mm + len(sizes)) % 16 else "f16", seed=len(sizes))


@pytest.mark.parametrize("sizes", [[900], [1313], [5000, 3], [0, 2000, 17, 1500], [1300, 1301]], ids=lambda s: f"{len(s)}x{max(s)}_{sum(s)}")
@pytest.mark.parametrize("mm,n", [(8, 8), (264, 136), (64, 520), (200, 200), (512, 256)])
def test_sums_few_tiles(m, sizes, mm, n):
    _check_sums(m, sizes, mm, n, "bf16" if (mm + len(sizes)) % 16 else "f16", pad=70, start=5, extra=(0, 8, 8), seed=len(sizes))


def test_sums_strided_padded(m):
    _check_sums(m, [33, 0, 20], 136, 264, "f16", pad=19, start=5, extra=(8, 16, 24), seed=3)
    _check_sums(m, [233, 0, 120, 1], 264, 72, "bf16", pad=70, start=65, extra=(0, 8, 16), seed=4)


@pytest.mark.parametrize("groups", [256, 1024])
def test_sums_many_groups(m, groups):
    r = random.Random(groups)
    _check_sums(m, [r.choice((0, 1, 2, 40, 100)) for _ in range(groups)], 72, 136, "bf16", seed=groups)


# ------------------------------------------------------------------ adapters

def _check_adapters(m, sizes, none, n, k, rank, dtype, order=True, scaled=True, in_place=False, extra=(0, 0, 0), ints=True, start=0, seed=0):
    t, rows, groups = TD[dtype], sum(sizes) + none + start, len(sizes)
    g = torch.Generator(device="cuda").manual_seed(seed + 9)
    if ints:
        x, base = _ints(seed, rows, k, dtype=t), _ints(seed + 1, rows, n, dtype=t, most=9)
        a, b = _ints(seed + 2, groups, rank, k, dtype=t, most=1), _ints(seed + 3, groups, n, rank, dtype=t, most=1)
        scales = (torch.randint(1, 5, (groups,), generator=g, device="cuda") / 2).float() if scaled else None
    else:
        def normal(*shape, scale=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * scale).to(t)
        x, base, a, b = normal(rows, k), normal(rows, n), normal(groups, rank, k, scale=k**-0.5), normal(groups, n, rank, scale=0.3)
        scales = torch.rand(groups, generator=g, device="cuda") if scaled else None
    x, base = _pitched(x, extra[0]), _pitched(base, extra[1])
    out = base if in_place else _pitched(torch.full((rows, n), -77.0, dtype=t, device="cuda"), extra[2])
    offsets, at = _offsets(sizes, start), np.concatenate([[0], np.cumsum(sizes)]) + start
    perm = torch.randperm(rows, generator=g, device="cuda") if order else torch.arange(rows, device="cuda")
    want, error = base.double(), torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    for e in range(groups):
        r = perm[at[e]:at[e + 1]]
        s = scales[e].double() if scaled else 1.0
        u, up = x[r].double() @ a[e].double().T, b[e].double().T
        want[r] += s * (u @ up)
        # u is off by its sum's 2^-20 sum |x a| (above) and by its pair's 2^-16 of the row's largest, and the
        # second sum by 2^-20 sum |u b|
        off = 2.0**-20 * (x[r].double().abs() @ a[e].double().abs().T) + 2.0**-16 * u.abs().amax(-1, keepdim=True)
        error[r] = s * ((off + 2.0**-20 * u.abs()) @ up.abs())
    op = m.Adapters(groups, n, k, rank, dtype=_code(m, dtype))
    op.run(x, a, b, offsets, perm.int() if order else None, base, out, scales=scales)
    assert op.sync_status() == m.GEMM_OK
    if ints:
        # u below 2^15 in magnitude is held exactly by the pair: 8 + 8 bits (bf16) or 11 + 11 of the row's largest
        assert torch.equal(out, want.to(t)), (out != want.to(t)).nonzero()[:5]
    else:
        # one addition in fp32 (2^-24 of the sum) and the result's half step, of a value that is off already
        half = torch.finfo(t).eps / 2
        tolerance = error + (want.abs() + error) * (half + 2.0**-23)
        assert ((out.double() - want).abs() <= tolerance).all(), ((out.double() - want).abs() - tolerance).max()


@pytest.mark.parametrize("sizes,none", [([1], 0), ([0, 1, 0, 0], 0), ([1, 2, 1, 0, 1], 3), ([8, 9, 7], 1), ([1] * 60, 4), ([0, 0], 5),
                                        ([33, 0, 64, 200], 7), ([700, 300], 0), ([5] * 150, 50), ([3000], 0), ([1] * 400, 1)])
@pytest.mark.parametrize("n,k,rank", [(8, 8, 8), (136, 72, 16), (1000, 2056, 24), (4096, 512, 64), (264, 1024, 128)])
def test_adapters(m, sizes, none, n, k, rank):
    i = len(sizes) + rank
    _check_adapters(m, sizes, none, n, k, rank, "bf16" if i % 2 else "f16", order=i % 3 > 0, scaled=i % 5 > 0, in_place=i % 4 == 0, seed=i)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rank", [8, 40, 64, 88])
def test_adapters_normal(m, dtype, rank):
    _check_adapters(m, [1, 0, 30, 2], 3, 520, 1032, rank, dtype, ints=False, seed=rank)
    _check_adapters(m, [100, 60, 0], 9, 520, 1032, rank, dtype, ints=False, order=False, seed=rank + 1)


# (every form of the operator, whatever the sizes would choose; with fewer blocks than CTAs another one would be taken)
FORMS = [(form, n, k, rank) for form in (0, 1, 2, 4, 8)
         for n, k, rank in ((8, 8, 8), (136, 72, 16), (1000, 328, 24), (520, 512, 64), (264, 200, 72), (392, 1024, 128), (1096, 1032, 48))
         if k >= 64 * form and n >= 128 * form]


@pytest.mark.parametrize("sizes,none", [([5000], 0), ([2600, 0, 2500], 60), ([200] * 40, 0), ([1, 6000, 17, 129, 128], 1), ([300, 33], 0),
                                        ([1000, 1, 700, 64], 500), ([0, 3], 2)], ids=lambda v: f"{len(v)}x{max(v)}" if isinstance(v, list) else str(v))
@pytest.mark.parametrize("form,n,k,rank", FORMS)
def test_adapters_forms(m, form, sizes, none, n, k, rank, monkeypatch):
    monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", str(form))
    i = len(sizes) + rank // 8
    _check_adapters(m, sizes, none, n, k, rank, "bf16" if i % 2 else "f16", order=i % 3 > 0, scaled=i % 5 > 0, in_place=i % 4 == 0, seed=i)
    _check_adapters(m, sizes, none, n, k, rank, "f16" if i % 2 else "bf16", order=i % 3 == 0, in_place=i % 4 == 1, extra=(8, 16, 16 if i % 4 == 1 else 24), start=11, seed=i + 1)


@pytest.mark.parametrize("sizes,none", [([5000], 0), ([200] * 40, 0), ([1, 16000, 17, 129, 128], 1), ([1000, 1, 700, 64], 500)],
                         ids=lambda v: f"{len(v)}x{max(v)}" if isinstance(v, list) else str(v))
@pytest.mark.parametrize("n,k,rank", [(4104, 2056, 64), (2048, 4096, 48), (3000, 2880, 128)])
def test_adapters_many_rows(m, sizes, none, n, k, rank):
    i = len(sizes) + rank // 8
    _check_adapters(m, sizes, none, n, k, rank, "bf16" if i % 2 else "f16", order=i % 3 > 0, seed=i)


# (every height of a tile of the form for few rows that there is, alone and in clusters: those of few tiles)
@pytest.mark.parametrize("sizes,none", [([1], 0), ([17, 0, 33, 8], 5), ([700, 300], 0), ([9] * 150, 50), ([5000, 1], 31)],
                         ids=lambda v: f"{len(v)}x{max(v)}" if isinstance(v, list) else str(v))
@pytest.mark.parametrize("height,n,k,rank", [(h, n, k, rank) for n, k, rank in ((136, 72, 16), (1000, 2056, 24), (4096, 512, 64), (264, 1032, 128))
                                             for h in (8, 16, 32) if (rank, h) not in ((64, 32), (128, 16))])
def test_adapters_heights(m, height, sizes, none, n, k, rank, monkeypatch):
    monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", "0")
    monkeypatch.setenv("LGT_GEMM_ADAPTERS_ROWS", str(height))
    i = len(sizes) + height // 8 + rank // 8
    _check_adapters(m, sizes, none, n, k, rank, "bf16" if i % 2 else "f16", order=i % 3 > 0, scaled=i % 5 > 0, in_place=i % 4 == 0, seed=i)
    _check_adapters(m, sizes, none, n, k, rank, "f16" if i % 2 else "bf16", ints=False, order=i % 3 == 0, extra=(8, 16, 24), start=11, seed=i + 1)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rank", [8, 64, 88])
@pytest.mark.parametrize("form", [0, 1, 4])
def test_adapters_forms_normal(m, dtype, rank, form, monkeypatch):
    monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", str(form))
    _check_adapters(m, [4000, 1500], 9, 520, 1032, rank, dtype, ints=False, order=rank == 64, seed=rank)


def test_adapters_strided(m):
    _check_adapters(m, [3, 0, 20], 2, 264, 136, 16, "f16", extra=(8, 16, 24), start=4, seed=1)
    _check_adapters(m, [200, 111, 300], 50, 264, 136, 32, "bf16", extra=(0, 8, 16), order=False, start=7, seed=2)
    _check_adapters(m, [40, 1], 50, 264, 136, 32, "bf16", extra=(8, 8, 8), in_place=True, seed=2)
