"""CPU tests of the serving operators' binding: what it looks at before it calls the library."""
import ctypes
import importlib.machinery
import importlib.util
import os
import shutil

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    import helpers
    m = helpers.lib()
    m._with_torch()
    return m


def _cache_attention(lib, batch, grow):
    """A CacheAttention as its constructor leaves it, without a device; `grow` in the place of its growth."""
    op = object.__new__(lib.CacheAttention)
    op.q_heads, op.k_heads, op.head_dim, op.page_size = 4, 2, 64, 16
    op.dtype, op.scale, op.code, op.batch = torch.float16, 0.0, lib.GEMM_F16, batch
    op.handle = (op.dtype, 4, 2, 64, 16, op.code, 0.0, 1 << 20, 1 << 20, batch, 0)
    op._grow = grow
    return op


@pytest.mark.parametrize("bad", ["host", "type", "shape", "table", "lengths"])
def test_refused_calls_do_not_grow_the_workspace(lib, bad):
    """A call that is refused anyway neither waits for the device nor allocates."""
    def grow(batch):
        raise AssertionError(f"grown to {batch}")
    op = _cache_attention(lib, 2, grow)
    c = lib.attn_cache_t(1 << 20, 1 << 20, 1 << 20, 1 << 20, 4, 16, 2, 64)

    class Cache:
        k_heads, head_dim, page_size, handle = 2, 64, 16, (ctypes.addressof(c), 2, 64, 0)
    n = 100
    q = torch.zeros(n, 4, 32 if bad == "shape" else 64, dtype=torch.float32 if bad == "type" else torch.float16)
    table, lengths = torch.zeros(n - (bad == "table"), 3, dtype=torch.int32), torch.zeros(n, dtype=torch.int64 if bad == "lengths" else torch.int32)
    with pytest.raises(ValueError):
        op.run(q, Cache, table, lengths, torch.zeros(n, 4, 64, dtype=torch.float16))
    assert op.batch == 2


class Tensor:
    """What the binding asks of a tensor, on the GPU numbered `device`."""

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self.is_cuda, self.device = tuple(shape), dtype, device >= 0, device

    def stride(self):
        s = [1]
        for n in self.shape[:0:-1]:
            s.append(s[-1] * n)
        return tuple(reversed(s))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def get_device(self):
        return self.device

    def __len__(self):
        return self.shape[0]


@pytest.fixture
def binding(lib, tmp_path):
    """A copy of the binding, with state of its own, whose library counts calls; `now` is the current device."""
    path = shutil.copy(lib._BINDING_PATH, tmp_path / "copied_binding.so")
    spec = importlib.util.spec_from_loader("_binding", importlib.machinery.ExtensionFileLoader("_binding", str(path)))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)

    class State:
        now, streams, calls = 0, [], []
    state = State()
    state.streams, state.calls = [], []

    def stand_in(name):
        f = ctypes.CFUNCTYPE(ctypes.c_int, *getattr(lib._lib, name).argtypes)(lambda *a: state.calls.append((name, a[-1])) or 0)
        state.__dict__.setdefault("keep", []).append(f)
        return ctypes.cast(f, ctypes.c_void_p).value

    def stream_of(device):
        state.streams.append(device)
        return 1000 + device
    module.setup(*(stand_in(n) for n in ("attn_rope_run", "attn_prompt_run", "attn_cache_write", "attn_cache_read", "attn_cache_attend")),
                 lambda: state.now, stream_of, torch.int32, torch.float16, torch.bfloat16)
    state.module = module
    return state


def _calls(lib, batch=4, kept=0):
    """Each operator's arguments before the stream, and the places of its tensors; `kept` is the device of caches and workspaces."""
    h, i = torch.float16, torch.int32
    c = lib.attn_cache_t(1 << 20, 1 << 20, 1 << 20, 1 << 20, 4, 16, 2, 64)
    cache = (ctypes.addressof(c), 2, 64, kept)
    q, k = (3, 4, 64), (3, 2, 64)
    return c, {
        "rope": [(0, h, 4, 2, 64), *(Tensor(s, t) for s, t in ((q, h), (k, h), ((3,), i), (q, h), (k, h), ((64,), h), ((64,), h)))],
        "prompt": [(0, h, 4, 2, 64), *(Tensor(s, t) for s, t in ((q, h), (k, h), (k, h), ((2,), i), ((2,), i), (q, h)))],
        "cache_write": [cache, *(Tensor(s, t) for s, t in ((k, h), (k, h), ((3,), i)))],
        "cache_read": [cache, *(Tensor(s, t) for s, t in ((k, h), (k, h), ((3,), i)))],
        "attend": [(h, 4, 2, 64, 16, lib.GEMM_F16, 0.0, 1 << 20, 1 << 20, batch, kept), cache,
                   *(Tensor(s, t) for s, t in ((q, h), ((3, 5), i), ((3,), i), (q, h)))],
    }


NAMES = ("rope", "prompt", "cache_write", "cache_read", "attend")


@pytest.mark.parametrize("name", NAMES)
def test_calls_take_the_current_stream_of_their_device(lib, binding, name):
    for device in (0, 1):
        c, calls = _calls(lib, kept=device)
        args = calls[name]
        for x in args:
            if isinstance(x, Tensor):
                x.device = device
        binding.now, f = device, getattr(binding.module, name)
        assert f(*args, None) == 0 and binding.calls[-1][1] == 1000 + device
        assert f(*args, 77) == 0 and binding.calls[-1][1] == 77
        assert f(*args, 0) == 0 and binding.calls[-1][1] is None
        assert binding.streams == list(range(device + 1)) and len(binding.calls) == 3 * (device + 1)


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(lib, binding, name):
    """One of them elsewhere, or all of them where the current device is not: the library is not called."""
    c, calls = _calls(lib)
    args, f = calls[name], getattr(binding.module, name)
    tensors = [x for x in args if isinstance(x, Tensor)]
    for x in tensors:
        for other in (1, -1):
            x.device, x.is_cuda = other, other >= 0
            assert f(*args, None) == -1 and f(*args, 77) == -1, (name, args.index(x), other)
        x.device, x.is_cuda = 0, True
    for x in tensors:
        x.device = 1
    assert f(*args, None) == -1 and f(*args, 77) == -1
    binding.now = 1  # (the cache, or the workspace, is still on device 0)
    assert (f(*args, None) == 0) == (name in ("rope", "prompt"))
    for x in tensors:
        x.device = 0
    assert f(*args, None) == -1 and f(*args, 77) == -1
    assert len(binding.calls) == (name in ("rope", "prompt"))


def test_a_larger_batch_is_told_from_a_refused_call(lib, binding):
    c, calls = _calls(lib, batch=2)
    args = calls["attend"]
    assert binding.module.attend(*args, None) == -2
    args[2].dtype = torch.bfloat16
    assert binding.module.attend(*args, None) == -1
    args[2].dtype, binding.now = torch.float16, 1
    assert binding.module.attend(*args, None) == -1 and not binding.calls


def test_the_refusal_names_the_device(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = Tensor((3, 2, 64), torch.float16, 1)
    with pytest.raises(ValueError, match="k is on cuda:1, the current device is cuda:0"):
        lib._refuse("attn_cache_write", -1, ("k", x, x.shape, x.dtype, True))
    x.device = 0
    with pytest.raises(ValueError, match="the cache is on cuda:2"):
        lib._refuse("attn_cache_write", -1, ("k", x, x.shape, x.dtype, True), kept=(("the cache", 2),))


def test_a_cache_is_on_one_device(lib):
    made = [torch.uint8] * 4
    k, v, ke, ve = (Tensor((2, 2, 16, 64)[: 4 - (i > 1)], t) for i, t in enumerate(made))
    for x in (k, v, ke, ve):
        x.dim = lambda x=x: len(x.shape)
    assert lib.KVCache(k, v, ke, ve).handle[3] == 0
    for x in (v, ke, ve):
        x.device = 1
        with pytest.raises(ValueError, match="another device"):
            lib.KVCache(k, v, ke, ve)
        x.device = 0


@pytest.fixture
def builder(lib, tmp_path, monkeypatch):
    """build.py over an output folder of its own and one small source."""
    path = os.path.join(os.path.dirname(lib.__file__), "build.py")
    spec = importlib.util.spec_from_file_location("build_under_test", path)
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    monkeypatch.setattr(b, "OUT_DIR", str(tmp_path))
    for name in ("LIB", "BINDING"):
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name))))
    monkeypatch.setattr(b, "SOURCES", ["noalloc.cu"])
    return b


@pytest.mark.parametrize("missing", ["headers", "compiler"])
def test_the_library_builds_where_the_binding_cannot(builder, monkeypatch, capfd, missing):
    """Products, the reduction and the dense attention go by ctypes and need neither."""
    with monkeypatch.context() as without:
        if missing == "headers":
            without.setattr(builder.sysconfig, "get_paths", lambda: {"include": "/nowhere"})
        else:
            which = shutil.which
            without.setattr(builder.shutil, "which", lambda x: "/nowhere/gcc" if x == "gcc" else which(x))
        open(builder.BINDING, "w").close()  # (one from before, of other sources)
        assert builder.build(force=True) == builder.LIB
        assert os.path.exists(builder.LIB) and not os.path.exists(builder.BINDING)
        assert "binding.c does not compile" in capfd.readouterr().err
    # where it can be built it is, by itself
    built = os.path.getmtime(builder.LIB)
    builder.build()
    assert os.path.exists(builder.BINDING) and os.path.getmtime(builder.LIB) == built
    assert capfd.readouterr().err == ""


def test_prompt_calls_without_a_plan(lib):
    for name in ("attn_prompt_withhold_load", "attn_prompt_sync_status"):
        args = [None] * len(getattr(lib._lib, name).argtypes)
        assert getattr(lib._lib, name)(*args) == lib.GEMM_ERR_INVALID_ARG
    assert lib._lib.attn_prompt_destroy(None) == lib.GEMM_OK


def test_a_missing_binding_is_said(lib, monkeypatch):
    monkeypatch.setattr(lib, "_BINDING_PATH", "/nowhere/_binding.so")
    with pytest.raises(ImportError, match="headers"):
        lib._with_torch()


def test_the_binding_is_of_one_interpreter(lib, monkeypatch):
    """Built and looked for under this interpreter's suffix, so that another one's is missing, not loaded."""
    import sysconfig
    here = sysconfig.get_config_var("EXT_SUFFIX")
    assert sysconfig.get_config_var("SOABI") in here
    folder = os.path.dirname(lib.__file__)

    def paths():
        found = []
        for name, attribute in (("build", "BINDING"), ("__init__", "_BINDING_PATH")):
            spec = importlib.util.spec_from_file_location(f"read_{name}", os.path.join(folder, f"{name}.py"))
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            found.append(getattr(module, attribute))
        return found
    assert paths() == [os.path.join(folder, "_lib", "_binding" + here)] * 2 and os.path.exists(paths()[0])
    monkeypatch.setattr(importlib.machinery, "EXTENSION_SUFFIXES", [".cpython-399-other.so"])
    assert paths() == [os.path.join(folder, "_lib", "_binding.cpython-399-other.so")] * 2
