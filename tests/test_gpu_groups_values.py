"""Operators over groups of rows on the GPU where values are far from ordinary."""
import pytest
import torch

from helpers import lib
from test_gpu_groups import TD, _code, _offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    return lib()


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
