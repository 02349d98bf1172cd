"""CPU tests of the serving operators' binding: what it looks at before it calls the library."""
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
    op.handle = (op.dtype, 4, 2, 64, 16, op.code, 0.0, 1 << 20, 1 << 20, batch)
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
        import ctypes
        address, k_heads, head_dim, page_size = ctypes.addressof(c), 2, 64, 16
    n = 100
    q = torch.zeros(n, 4, 32 if bad == "shape" else 64, dtype=torch.float32 if bad == "type" else torch.float16)
    table, lengths = torch.zeros(n - (bad == "table"), 3, dtype=torch.int32), torch.zeros(n, dtype=torch.int64 if bad == "lengths" else torch.int32)
    with pytest.raises(ValueError):
        op.run(q, Cache, table, lengths, torch.zeros(n, 4, 64, dtype=torch.float16))
    assert op.batch == 2
