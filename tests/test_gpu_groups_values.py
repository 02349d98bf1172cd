"""Operators over groups of rows on the GPU where values are far from ordinary:
adapters of infinite weights, rows of which one value is infinite, products whose
factors pass the types' ends while the result does not; sums beside rows of infinities.
Infinities and NaN have to be where the definition in 64 bits has them.

Finite results of adapters: u is off by its sum's 2^-20 sum |x a| and by its pair's 2^-16 of the
row's largest finite value, the second sum by 2^-20 sum |u b|, the result by one fp32
rounding (2^-23 is ample) and half a step of its type; a result below the least normal
value by half a step there."""
import pytest
import torch

from helpers import lib
from test_gpu_groups import TD, _code, _offsets

pytestmark = pytest.mark.gpu

# rows of the groups, and the form: the one for few rows, the one for many with 1, 2 and 4 CTAs a tile
CALLS = [([5, 0, 3], 0), ([90, 0, 133], 0), ([90, 0, 133], 1), ([90, 0, 133], 2), ([90, 0, 133], 4)]
N, K = 520, 256


@pytest.fixture(scope="module")
def m():
    return lib()


def _check(m, monkeypatch, form, sizes, x, a, b, base, scales=None):
    """One call against the definition, value by value in 64 bits."""
    monkeypatch.setenv("LGT_GEMM_ADAPTERS_FORM", str(form))
    t, dtype = x.dtype, "f16" if x.dtype is torch.float16 else "bf16"
    offsets, out = _offsets(sizes), torch.full_like(base, -77.0)
    op = m.Adapters(a.shape[0], b.shape[1], x.shape[1], a.shape[1], dtype=_code(m, dtype))
    op.run(x, a, b, offsets, None, base, out, scales=scales)
    assert op.sync_status() == m.GEMM_OK
    at = offsets.tolist()
    for g in range(len(sizes)):
        r = slice(at[g], at[g + 1])
        if at[g] == at[g + 1]:
            continue
        s = scales[g].double() if scales is not None else torch.ones((), dtype=torch.float64, device="cuda")
        u = (x[r, None].double() * a[g, None].double()).sum(-1)
        up = b[g].double()
        want = base[r].double() + s * (u[:, None] * up[None]).sum(-1)
        got = out[r].double()
        there = want.isfinite()
        # (a finite value beyond the type's range becomes an infinity)
        want_t = want.to(t).double()
        there &= want_t.isfinite()
        assert torch.equal(got.isnan(), want.isnan()), (g, (got.isnan() != want.isnan()).nonzero()[:5])
        assert torch.equal(got[~there & ~want.isnan()], want_t[~there & ~want.isnan()]), g
        finite = torch.where(u.isfinite(), u, 0.0)
        off = 2.0**-20 * (x[r].double().abs() @ a[g].double().abs().nan_to_num(posinf=0.0).T) + 2.0**-16 * finite.abs().amax(-1, keepdim=True)
        error = s.abs() * ((off + 2.0**-20 * finite.abs()) @ up.abs().nan_to_num(posinf=0.0).T)
        half = torch.finfo(t).eps / 2
        tolerance = error + (want.abs() + error) * (half + 2.0**-23) + torch.finfo(t).smallest_normal * half
        assert ((got - want).abs() <= tolerance)[there].all(), (g, ((got - want).abs() / tolerance)[there].max())


def _rows(sizes, t, g):
    """Rows of x with one or two values of 1: each u is a value of A, which the type holds, or the sum of two."""
    rows = sum(sizes)
    x = torch.zeros(rows, K, dtype=t, device="cuda")
    for i in range(2):
        x[torch.arange(rows, device="cuda"), torch.randint(0, K, (rows,), generator=g, device="cuda")] = 1
        if i == 0:
            keep = x[::2].clone()
    x[::2] = keep
    return x


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sizes,form", CALLS)
@pytest.mark.parametrize("rank", [8, 24, 80])
def test_infinite_weights_of_an_adapter(m, sizes, form, dtype, rank, monkeypatch):
    """A column of B with an infinite value gives infinities of the sign that the definition gives, and NaN where
    u is 0 or two of them are opposed."""
    t, groups = TD[dtype], len(sizes)
    g = torch.Generator(device="cuda").manual_seed(rank + form)
    x = _rows(sizes, t, g)
    a = torch.randn(groups, rank, K, generator=g, device="cuda").to(t)
    a[:, 1] = 0
    a[:, 3] = (a[:, 3].float() * 2.0**-14).to(t)  # far below the others of its row
    a[:, 4] = (a[:, 4].float() * (2.0**-24 if dtype == "f16" else 2.0**-90)).to(t)
    a[:, 5] = (a[:, 5].float() * 2.0**8).to(t)
    b = (torch.randn(groups, N, rank, generator=g, device="cuda") * 0.3).to(t)
    for i in range(rank):  # of each value of u, columns where its weight is infinite
        b[:, i * 5::rank * 5 + 1, i] = float("inf")
        b[:, i * 5 + 2::rank * 5 + 1, i] = -float("inf")
    b[:, 3::17, 0], b[:, 3::17, 2] = float("inf"), float("inf")
    base = torch.randn(x.shape[0], N, generator=g, device="cuda").to(t)
    _check(m, monkeypatch, form, sizes, x, a, b, base)
    _check(m, monkeypatch, form, sizes, x, a, b, base, scales=torch.tensor([-2.0, 1.0, 0.5], device="cuda"))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sizes,form", CALLS)
def test_an_infinite_value_beside_large_ones(m, sizes, form, dtype, monkeypatch):
    """One value of u is infinite, the others are finite, in fp16 above the largest that the type holds."""
    t, groups, rank = TD[dtype], len(sizes), 16
    g = torch.Generator(device="cuda").manual_seed(form)
    x = torch.zeros(sum(sizes), K, dtype=t, device="cuda")
    x[:, 0], x[:, 1] = 1, 4
    x[::3, 0] = -1
    x[1::4, 0] = 0  # (no number: 0 times an infinity)
    a = torch.zeros(groups, rank, K, dtype=t, device="cuda")
    a[:, 0, 0] = float("inf")
    a[:, 1, 1], a[:, 2, 1] = 30000, -50000
    b = torch.randint(-2, 3, (groups, N, rank), generator=g, device="cuda").to(t)
    base = torch.randn(x.shape[0], N, generator=g, device="cuda").to(t)
    _check(m, monkeypatch, form, sizes, x, a, b, base)


ENDS = {
    # x, A, B, scale: the first product's and the scale's magnitudes together pass fp32's range, the result does not
    "scaled up": ("bf16", 2.0**63, 2.0**61, 2.0**-125, 2.0**9),
    "scaled down": ("bf16", 2.0**-60, 2.0**-58, 2.0**120, -(2.0**-30)),
    "a scale near zero": ("bf16", 2.0**60, 2.0**40, 2.0**30, 2.0**-140),
    "a large scale": ("bf16", 2.0**-60, 2.0**-50, 2.0**-10, 2.0**125),
    "a scale of zero": ("bf16", 2.0**63, 2.0**61, 2.0**-125, 0.0),
    "an infinite scale": ("bf16", 1.0, 1.0, 1.0, float("inf")),
    "half, scaled up": ("f16", 2.0**12, 2.0**12, 2.0**-20, 2.0**115),
    "half, scaled down": ("f16", 2.0**-12, 2.0**-10, 2.0**10, 2.0**14),
    "half, a scale near zero": ("f16", 2.0**12, 2.0**12, 2.0**10, 2.0**-140),
}


@pytest.mark.parametrize("sizes,form", CALLS)
@pytest.mark.parametrize("end", ENDS)
def test_factors_past_the_range_of_fp32(m, sizes, form, end, monkeypatch):
    """u, the scale and B, whose product is a moderate number, in any distribution; columns of zeros among B's give base."""
    dtype, *size, scale = ENDS[end]
    t, groups, rank = TD[dtype], len(sizes), 16
    g = torch.Generator(device="cuda").manual_seed(form)
    x = (_rows(sizes, t, g).float() * size[0]).to(t)
    a = ((torch.rand(groups, rank, K, generator=g, device="cuda") + 0.5) * size[1]).to(t)
    b = ((torch.rand(groups, N, rank, generator=g, device="cuda") + 0.5) * size[2]).to(t)
    b[:, ::7] = 0
    b[:, 1::5] *= -1
    base = torch.randn(x.shape[0], N, generator=g, device="cuda").to(t)
    _check(m, monkeypatch, form, sizes, x, a, b, base, scales=torch.full((groups,), scale, device="cuda"))


@pytest.mark.parametrize("sizes,form", CALLS)
@pytest.mark.parametrize("rank", [16, 128])
def test_weights_near_the_types_end(m, sizes, form, rank, monkeypatch):
    """The sum over the rank of large weights passes fp32's range before the row's power of two brings it back."""
    t, groups = torch.bfloat16, len(sizes)
    g = torch.Generator(device="cuda").manual_seed(form)
    x = (_rows(sizes, t, g).float() * 2.0**-40).to(t)
    a = ((torch.rand(groups, rank, K, generator=g, device="cuda") + 0.5) * 2.0**-40).to(t)
    b = ((torch.rand(groups, N, rank, generator=g, device="cuda") * 0.4 + 0.5) * 2.0**128).to(t)
    base = torch.randn(x.shape[0], N, generator=g, device="cuda").to(t)
    _check(m, monkeypatch, form, sizes, x, a, b, base)


@pytest.mark.parametrize("sizes,form", CALLS)
def test_first_products_below_the_normal_values(m, sizes, form, monkeypatch):
    """u is less than 2^-126, where fp32 and bf16 have fewer bits: it comes in whole steps of 2^-149 here, as the sums
    of fp32 hold them, and the second product takes them up without a further loss."""
    t, groups, rank = torch.bfloat16, len(sizes), 16
    g = torch.Generator(device="cuda").manual_seed(form)
    x = torch.zeros(sum(sizes), K, dtype=t, device="cuda")
    x[:, 5] = 2.0**-80
    a = torch.zeros(groups, rank, K, dtype=t, device="cuda")
    a[:, :, 5] = (torch.randint(1, 256, (groups, rank), generator=g, device="cuda").float() * 2.0**-69).to(t)
    b = (torch.randn(groups, N, rank, generator=g, device="cuda") * 2.0**40).to(t)
    base = torch.zeros(x.shape[0], N, dtype=t, device="cuda")
    _check(m, monkeypatch, form, sizes, x, a, b, base, scales=torch.full((groups,), 2.0**96, device="cuda"))


@pytest.mark.parametrize("sizes,form", CALLS)
def test_everything_large_but_the_weights(m, sizes, form, monkeypatch):
    """u and the scale near the end of the range, whose weights have the least values of bf16, or are 0."""
    t, groups, rank = torch.bfloat16, len(sizes), 16
    g = torch.Generator(device="cuda").manual_seed(form)
    x = (_rows(sizes, t, g).float() * 2.0**63).to(t)
    a = ((torch.rand(groups, rank, K, generator=g, device="cuda") * 0.4 + 0.5) * 2.0**63).to(t)
    b = (torch.randint(-1, 2, (groups, N, rank), generator=g, device="cuda").double() * 2.0**-132).to(t)
    base = torch.randn(x.shape[0], N, generator=g, device="cuda").to(t)
    _check(m, monkeypatch, form, sizes, x, a, b, base, scales=torch.full((groups,), 1.5 * 2.0**127, device="cuda"))


@pytest.mark.parametrize("sizes,form", CALLS)
def test_everything_large_but_the_scale(m, sizes, form, monkeypatch):
    """u and B near the end of the range under a scale below the normal values."""
    t, groups, rank = torch.bfloat16, len(sizes), 16
    g = torch.Generator(device="cuda").manual_seed(form)
    x = (_rows(sizes, t, g).float() * 2.0**63).to(t)
    a = ((torch.rand(groups, rank, K, generator=g, device="cuda") + 0.5) * 2.0**62).to(t)
    b = ((torch.rand(groups, N, rank, generator=g, device="cuda") * 0.4 + 0.5) * 2.0**128).to(t)
    base = torch.randn(x.shape[0], N, generator=g, device="cuda").to(t)
    _check(m, monkeypatch, form, sizes, x, a, b, base, scales=torch.full((groups,), 2.0**-145, device="cuda"))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mm,n", [(264, 200), (136, 520), (512, 1024)])
def test_sums_between_groups_of_infinities(m, dtype, mm, n):
    """Pairs, where each CTA clears its part of what lies behind a group's last whole step: every second group's rows
    are infinite or no numbers, and no call out of many lets them into a neighbour's sums.  Whole numbers: exact."""
    t = TD[dtype]
    g = torch.Generator(device="cuda").manual_seed(mm)
    sizes = [1 + (i * 29) % 83 for i in range(90)]
    offsets = _offsets(sizes)
    at = offsets.tolist()
    a, b = (torch.randint(-3, 4, (sum(sizes), c), generator=g, device="cuda").to(t) for c in (mm, n))
    for i in range(1, 90, 2):
        a[at[i]:at[i + 1]] = float("inf") if i % 4 == 1 else float("nan")
        b[at[i]:at[i + 1]] = -float("inf")
    want = torch.stack([a[at[i]:at[i + 1]].double().T @ b[at[i]:at[i + 1]].double() for i in range(0, 90, 2)]).to(t)
    op, c = m.GroupedGemmK(90, mm, n, dtype=_code(m, dtype)), torch.empty(90, mm, n, dtype=t, device="cuda")
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(60):
        c.fill_(-77.0)
        op.run(a, b, offsets, c)
        bad += (c[::2] != want).sum()
    assert op.sync_status() == m.GEMM_OK and int(bad) == 0
    assert not c[1::2].isfinite().any()
