"""CPU tests of the operators over groups of rows: the refusals of their entry
points, what the binding looks at before it calls the library, and the split of a
group's rows into tiles, restated from its integer formulas.  No GPU work: every
call here is refused before a launch, or has nothing to do."""
import ctypes
import importlib.machinery
import importlib.util
import shutil

import numpy as np
import pytest
import torch

from test_serving_binding import Tensor


@pytest.fixture(scope="module")
def lib():
    import helpers
    m = helpers.lib()
    m._with_torch()
    return m


def _status(run, ok):
    def status(**kw):
        assert set(kw) <= set(ok)
        return run(*{**ok, **kw}.values(), None)
    return status


def test_row_groups_refuses(lib):
    bad, s = lib.GEMM_ERR_INVALID_ARG, _status(lib._lib.gemm_row_groups, dict(ids=1 << 20, rows=10, groups=4, offsets=1 << 21, order=1 << 22, places=1 << 23))
    assert s(rows=-1) == s(groups=0) == s(groups=1025) == bad
    assert s(ids=None) == s(offsets=None) == s(order=None) == bad
    assert s(order=1 << 20) == s(places=(1 << 22) + 36) == s(offsets=(1 << 20) + 4) == s(offsets=(1 << 23) - 16) == bad  # overlapping
    for name in ("ids", "offsets", "order", "places"):
        assert s(**{name: (1 << 24) + 2}) == lib.GEMM_ERR_ALIGNMENT
    assert s(rows=(1 << 30) + 1, order=1 << 40, places=1 << 41, offsets=1 << 42) == lib.GEMM_ERR_UNSUPPORTED


def _grouped(lib, **kw):
    a = dict(groups=4, form=lib.GEMM_GROUPED_M, M=0, N=64, K=128, b_layout=lib.GEMM_K_CONTIG, dtype=lib.GEMM_BF16)
    a.update(kw)
    return lib.gemm_grouped_create_status(lib.gemm_grouped_desc_t(*a.values()))


@pytest.mark.parametrize("kw", [dict(groups=0), dict(groups=1025), dict(form=2), dict(form=-1), dict(M=8), dict(N=0), dict(N=12), dict(N=-8),
                                dict(N=1 << 30), dict(K=0), dict(K=60), dict(b_layout=2), dict(dtype=3), dict(dtype=2),
                                dict(form=1, K=0, b_layout=1, M=0), dict(form=1, K=0, b_layout=1, M=12), dict(form=1, K=8, b_layout=1, M=8),
                                dict(form=1, K=0, b_layout=0, M=8)])
def test_grouped_refuses_descriptions(lib, kw):
    st, h = _grouped(lib, **kw)
    assert st == lib.GEMM_ERR_INVALID_ARG and not h


@pytest.mark.parametrize("along_k", [False, True])
def test_grouped_refuses_runs(lib, along_k):
    st, h = _grouped(lib, **(dict(form=1, M=128, K=0, b_layout=1) if along_k else {}))
    assert st == lib.GEMM_OK and h
    s = _status(lib._lib.gemm_grouped_run, dict(plan=h, A=1 << 20, lda=0, B=1 << 22, ldb=0, b_stride=0, offsets=1 << 24, rows=5, C=1 << 26, ldc=0, c_stride=0))
    bad = lib.GEMM_ERR_INVALID_ARG
    assert s(plan=None) == s(rows=-1) == s(A=None) == s(B=None) == s(C=None) == s(offsets=None) == bad
    assert s(lda=64) == s(lda=132) == s(lda=-128) == s(lda=1 << 40) == bad
    assert s(ldb=56) == s(ldb=130) == s(ldb=-8) == bad
    assert s(ldc=56) == s(ldc=68) == s(ldc=-64) == s(ldc=1 << 62) == bad
    if along_k:
        assert s(c_stride=64 * 127) == s(c_stride=64 * 128 + 4) == s(c_stride=-8) == s(c_stride=1 << 40) == bad
    else:
        assert s(b_stride=128 * 63) == s(b_stride=128 * 64 + 4) == s(b_stride=-8) == s(b_stride=1 << 40) == bad
        assert s(rows=0) == s(rows=0, A=None, C=None) == lib.GEMM_OK
    for name in ("A", "B", "C"):
        assert s(**{name: (1 << 28) + 8}) == lib.GEMM_ERR_ALIGNMENT
    assert s(offsets=(1 << 28) + 2) == lib.GEMM_ERR_ALIGNMENT
    assert s(rows=(1 << 30) + 1) == lib.GEMM_ERR_UNSUPPORTED
    assert lib._lib.gemm_grouped_sync_status(None, None) == bad and lib._lib.gemm_grouped_withhold_load(None) == bad
    assert lib._lib.gemm_grouped_destroy(h) == lib.GEMM_OK and lib._lib.gemm_grouped_destroy(None) == lib.GEMM_OK


@pytest.mark.parametrize("kw", [dict(groups=0), dict(groups=1025), dict(rank=0), dict(rank=4), dict(rank=20), dict(rank=136), dict(N=0), dict(N=12),
                                dict(K=4), dict(K=1 << 30), dict(dtype=2)])
def test_adapters_refuse_descriptions(lib, kw):
    d = {**dict(groups=3, rank=16, N=64, K=128, dtype=lib.GEMM_F16), **kw}
    st, h = lib.gemm_adapters_create_status(lib.gemm_adapters_desc_t(*d.values()))
    assert st == lib.GEMM_ERR_INVALID_ARG and not h


def test_adapters_refuse_runs(lib):
    st, h = lib.gemm_adapters_create_status(lib.gemm_adapters_desc_t(3, 16, 64, 128, lib.GEMM_F16))
    assert st == lib.GEMM_OK and h
    s = _status(lib._lib.gemm_adapters_run, dict(plan=h, x=1 << 20, xs=0, A=1 << 21, B=1 << 22, scales=1 << 23, offsets=1 << 24, order=1 << 25, rows=5,
                                                 base=1 << 26, bs=0, out=1 << 27, os=0))
    bad = lib.GEMM_ERR_INVALID_ARG
    for name in ("plan", "x", "A", "B", "offsets", "base", "out"):
        assert s(**{name: None}) == bad
    assert s(rows=-1) == s(xs=120) == s(xs=132) == s(bs=56) == s(bs=68) == s(os=60) == s(os=-64) == s(xs=1 << 40) == bad
    assert s(out=1 << 26, os=72) == bad  # in place, with another pitch
    for name in ("x", "A", "B", "base", "out"):
        assert s(**{name: (1 << 28) + 8}) == lib.GEMM_ERR_ALIGNMENT
    for name in ("scales", "offsets", "order"):
        assert s(**{name: (1 << 28) + 2}) == lib.GEMM_ERR_ALIGNMENT
    assert s(rows=(1 << 30) + 1) == lib.GEMM_ERR_UNSUPPORTED and s(rows=0, x=None, out=None) == lib.GEMM_OK
    assert lib._lib.gemm_adapters_destroy(h) == lib.GEMM_OK and lib._lib.gemm_adapters_destroy(None) == lib.GEMM_OK


def test_host_tensors_are_refused(lib):
    i, x = torch.zeros(5, dtype=torch.int32), torch.zeros(5, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        lib.row_groups(i, i[:3], i)
    with pytest.raises(ValueError):
        lib.row_groups(i, i[:1], i)
    with pytest.raises(ValueError):
        lib.GroupedGemm(4, 64, 64, dtype=lib.GEMM_F16).run(x, torch.zeros(4, 64, 64, dtype=torch.float16), i, x)
    with pytest.raises(ValueError):
        lib.GroupedGemmK(4, 64, 64, dtype=lib.GEMM_F16).run(x, x, i, torch.zeros(4, 64, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        lib.Adapters(4, 64, 64, 8, dtype=lib.GEMM_F16).run(x, torch.zeros(4, 8, 64, dtype=torch.float16), torch.zeros(4, 64, 8, dtype=torch.float16), i, None, x, x)
    with pytest.raises(lib.GemmError):
        lib.GroupedGemm(4, 60, 64)
    with pytest.raises(lib.GemmError):
        lib.Adapters(4, 64, 64, 12)


class Strided(Tensor):
    """A stand-in whose dimensions are `strides` apart."""

    def __init__(self, shape, dtype, strides, device=0):
        super().__init__(shape, dtype, device)
        self.strides = tuple(strides)

    def stride(self):
        return self.strides

    def is_contiguous(self):
        return False


@pytest.fixture
def binding(lib, tmp_path):
    """A copy of the binding whose library notes its arguments; `now` is the current device."""
    path = shutil.copy(lib._BINDING_PATH, tmp_path / "copied_binding.so")
    spec = importlib.util.spec_from_loader("_binding", importlib.machinery.ExtensionFileLoader("_binding", str(path)))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)

    class State:
        now, calls, keep = 0, [], []
    state = State()
    state.calls, state.keep = [], []

    def stand_in(name):
        f = ctypes.CFUNCTYPE(ctypes.c_int, *getattr(lib._lib, name).argtypes)(lambda *a: state.calls.append((name, a)) or 0)
        state.keep.append(f)
        return ctypes.cast(f, ctypes.c_void_p).value
    module.setup(*(stand_in(n) for n in ("attn_rope_run", "attn_prompt_run", "attn_cache_write", "attn_cache_read", "attn_cache_attend")),
                 lambda: state.now, lambda device: 1000 + device, torch.int32, torch.float16, torch.bfloat16)
    module.setup_groups(*(stand_in(n) for n in ("gemm_row_groups", "gemm_grouped_run", "gemm_adapters_run")), torch.float32)
    state.module = module
    return state


H, I, F = torch.float16, torch.int32, torch.float32


def _calls():
    return {
        "row_groups": [Tensor((7,), I), Tensor((5,), I), Tensor((7,), I), Tensor((7,), I)],
        "grouped": [(0, H, 4, 0, 64, 128, 1), Tensor((7, 128), H), Tensor((4, 64, 128), H), Tensor((5,), I), Tensor((7, 64), H)],
        "grouped_mn": [(0, H, 4, 0, 64, 128, 0), Tensor((7, 128), H), Tensor((4, 128, 64), H), Tensor((5,), I), Tensor((7, 64), H)],
        "grouped_k": [(0, H, 4, 32, 64, 0, 0), Tensor((7, 32), H), Tensor((7, 64), H), Tensor((5,), I), Tensor((4, 32, 64), H)],
        "adapters": [(0, H, 4, 64, 128, 16), Tensor((7, 128), H), Tensor((4, 16, 128), H), Tensor((4, 64, 16), H), Tensor((5,), I), Tensor((7,), I),
                     Tensor((7, 64), H), Tensor((7, 64), H), Tensor((4,), F)],
    }


NAMES = tuple(_calls())


@pytest.mark.parametrize("name", NAMES)
def test_binding_looks_at_every_tensor(binding, name):
    f = getattr(binding.module, name.split("_")[0] if name.startswith("grouped") else name)
    for device in (0, 1):
        args = _calls()[name]
        binding.now = device
        for x in args:
            if isinstance(x, Tensor):
                x.device = device
        assert f(*args, None) == 0 and binding.calls[-1][1][-1] == 1000 + device
        assert f(*args, 77) == 0 and binding.calls[-1][1][-1] == 77
    binding.now, done = 0, len(binding.calls)
    for i, x in enumerate(_calls()[name]):
        if not isinstance(x, Tensor):
            continue
        for change in ("device", "host", "type", "shape", "dims", "none at all"):
            args = _calls()[name]
            t = args[i]
            if change == "device":
                t.device = 1
            elif change == "host":
                t.device = -1
            elif change == "type":
                t.dtype = torch.float64
            elif change == "shape":
                # (the first tensor's rows and offsets' groups, for row_groups, decide the others')
                if name == "row_groups" and i == 1:
                    t.shape = (1,)
                else:
                    t.shape = (t.shape[0] + 1, *t.shape[1:]) if i != 1 or name == "row_groups" else (t.shape[0], *t.shape[1:-1], t.shape[-1] + 8)
            elif change == "dims":
                t.shape = (*t.shape, 1)
            else:
                args[i] = object()
            assert f(*args, None) == -1, (i, change)
        if len(x.shape) > 1:
            for strides in ([n + 1 for n in x.stride()], [*x.stride()[:-1], 2], [0, *x.stride()[1:]], [8, *x.stride()[1:]]):
                args = _calls()[name]
                args[i] = Strided(x.shape, x.dtype, strides)
                pitched = strides[-1] == 1 and strides[0] >= x.stride()[0] and (len(x.shape) == 2 or strides[1] >= x.stride()[1])
                if not pitched or (name == "adapters" and len(x.shape) == 3):
                    assert f(*args, None) == -1, (i, strides)
    assert len(binding.calls) == done
    binding.now = 1
    assert f(*_calls()[name], None) == -1  # tensors of another device than the current one
    with pytest.raises(TypeError):
        f(*_calls()[name])


def test_binding_passes_pitches(binding):
    m = binding.module
    args = _calls()["grouped"]
    args[1], args[2], args[4] = Strided((7, 128), H, (136, 1)), Strided((4, 64, 128), H, (64 * 144 + 8, 144, 1)), Strided((7, 64), H, (80, 1))
    assert m.grouped(*args, None) == 0
    assert binding.calls[-1][1][1:11] == (1 << 20, 136, 1 << 20, 144, 64 * 144 + 8, 1 << 20, 7, 1 << 20, 80, 0)
    args = _calls()["grouped_k"]
    args[1], args[2], args[4] = Strided((7, 32), H, (40, 1)), Strided((7, 64), H, (72, 1)), Strided((4, 32, 64), H, (32 * 72, 72, 1))
    assert m.grouped(*args, None) == 0
    assert binding.calls[-1][1][1:11] == (1 << 20, 40, 1 << 20, 72, 0, 1 << 20, 7, 1 << 20, 72, 32 * 72)
    # one row, one group: their strides say nothing
    args = _calls()["grouped"]
    args[1], args[4] = Strided((1, 128), H, (3, 1)), Strided((1, 64), H, (5, 1))
    assert m.grouped(*args, None) == 0 and binding.calls[-1][1][2] == 0 and binding.calls[-1][1][9] == 0
    args = _calls()["adapters"]
    args[5], args[8] = None, None
    assert m.adapters(*args, None) == 0
    assert binding.calls[-1][1][5:9] == (None, 1 << 20, None, 7)
    args = _calls()["row_groups"]
    args[3] = None
    assert m.row_groups(*args, None) == 0 and binding.calls[-1][1][1:3] == (7, 4) and binding.calls[-1][1][5] is None


def test_tiles_of_a_group_cover_its_rows_once():
    """Tiles as even as steps of 16 or 32 allow, none empty, none wider than the most."""
    rng = np.random.default_rng(0)
    for _ in range(3000):
        step = int(rng.choice([16, 32]))
        most = step * int(rng.integers(1, 256 // step + 1))
        length = int(rng.integers(1, 3000))
        tiles = -(-length // most)
        width = -(-(-(-length // tiles)) // step) * step
        ends = [min((i + 1) * width, length) for i in range(tiles)]
        assert width <= most and ends[-1] == length and (tiles - 1) * width < length


def test_tiles_in_bands_are_each_taken_once():
    """The order of a group's tiles (in bands of eight of the N side) names each of them once."""
    band = 8
    for p_tiles in (1, 2, 3, 7, 12, 32):
        for q_tiles in (1, 2, 5, 7, 8, 9, 15, 16, 17, 40):
            seen = set()
            for r in range(p_tiles * q_tiles):
                first, high = 0, q_tiles
                if q_tiles > band:
                    first = r // (p_tiles * band)
                    r -= first * (p_tiles * band)
                    high = min(band, q_tiles - first * band)
                p = r // high
                seen.add((p, first * band + r - p * high))
            assert seen == {(p, q) for p in range(p_tiles) for q in range(q_tiles)}


def test_reciprocals_of_a_band_divide_exactly():
    """n / d as the upper half of n times 2^32 / d, rounded up: exact for d up to 8 and n below 2^29, since the product
    is too large by less than n * d / 2^32 < 1 / d of a whole."""
    for d in range(2, 9):
        m = ((1 << 32) + d - 1) // d
        for near in list(range(0, 4096)) + [k * d for k in range(1 << 10, 1 << 26, 65537)] + [(1 << 29) - 1, (1 << 29) // d * d - 1]:
            for n in (near, max(near - 1, 0), near + 1 if near + 1 < 1 << 29 else near):
                assert n * m >> 32 == n // d


@pytest.mark.parametrize("values", [0, 1, 1026, 5000])
def test_a_number_of_groups_that_is_refused_is_named(lib, values):
    ids = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="1 to 1024 groups"):
        lib.row_groups(ids, torch.zeros(values, dtype=torch.int32), ids.clone())
