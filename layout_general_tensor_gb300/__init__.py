"""Python binding of the any-layout GEMM C ABI (``include/gemm.h``), the fp32
row reduction (``include/reduce.h``), the fused attention
(``include/attention.h``) and the operators of a serving attention layer
(``include/attn_rope.h``, ``include/attn_prompt.h``, ``include/attn_cache.h``).

Argument marshalling only: every function forwards to the entry point of the
same name in ``_lib/libgemm.so``; all arithmetic runs in the library's CUDA
kernels.  Importing this package fails loudly when the library has not been
built -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libgemm.so")
# (of this interpreter: the part in C goes by the layouts of one)
_BINDING_PATH = os.path.join(_HERE, "_lib", "_binding" + importlib.machinery.EXTENSION_SUFFIXES[0])

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_UNSUPPORTED = 2
GEMM_ERR_ALIGNMENT = 3
GEMM_ERR_WORKSPACE = 4
GEMM_ERR_CUDA = 5
GEMM_ERR_TIMEOUT = 6

GEMM_FLAG_DETERMINISTIC = 1
GEMM_FLAG_INT4_PREPACKED = 4
GEMM_FLAG_TEST_WITHHOLD_STAGE = 1 << 30

GEMM_K_CONTIG = 0
GEMM_MN_CONTIG = 1

GEMM_F16 = 0
GEMM_BF16 = 1
GEMM_INT4 = 2
GEMM_F32 = 3

ATTN_ROPE_HALF = 0
ATTN_ROPE_INTERLEAVED = 1

# Every entry point the headers under include/ declare.
EXPORTS = (
    "gemm_create", "gemm_workspace_size", "gemm_query", "gemm_run", "gemm_run_static_scratch",
    "gemm_sync_status", "gemm_destroy",
    "gemm_splitk_auto", "gemm_perm_fwd", "gemm_perm_inv", "gemm_perm_device", "gemm_magic_divmod_host",
    "gemm_magic_divmod_device", "gemm_status_string", "gemm_int4_prepack_bytes", "gemm_int4_prepack",
    "reduce_rows_workspace_size", "reduce_rows_f32",
    "attn_create", "attn_run", "attn_sync_status", "attn_destroy",
    "attn_rope_frequencies", "attn_rope_create", "attn_rope_run", "attn_rope_destroy",
    "attn_prompt_create", "attn_prompt_run", "attn_prompt_sync_status",
    "attn_prompt_withhold_load", "attn_prompt_destroy",
    "attn_cache_write", "attn_cache_read", "attn_cache_attend_workspace_size", "attn_cache_attend",
)


class gemm_desc_t(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("a_layout", ctypes.c_int32), ("b_layout", ctypes.c_int32),
        ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64), ("ldc", ctypes.c_int64),
        ("a_dtype", ctypes.c_int32), ("b_dtype", ctypes.c_int32), ("c_dtype", ctypes.c_int32),
        ("split_k", ctypes.c_int32), ("group_size", ctypes.c_int32), ("num_sms", ctypes.c_int32),
        ("flags", ctypes.c_int32),
    ]


class attn_desc_t(ctypes.Structure):
    _fields_ = [
        ("heads", ctypes.c_int32), ("seq_q", ctypes.c_int32), ("seq_k", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
    ]


class attn_rope_desc_t(ctypes.Structure):
    _fields_ = [
        ("q_heads", ctypes.c_int32), ("k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("eps", ctypes.c_float), ("magnitude", ctypes.c_float),
        ("base", ctypes.c_double), ("factor", ctypes.c_double), ("context", ctypes.c_double),
        ("low_turns", ctypes.c_double), ("high_turns", ctypes.c_double),
    ]


class attn_prompt_desc_t(ctypes.Structure):
    _fields_ = [
        ("q_heads", ctypes.c_int32), ("k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("causal", ctypes.c_int32), ("scale", ctypes.c_float),
    ]


class attn_cache_t(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p),
        ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("k_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
    ]


class gemm_info_t(ctypes.Structure):
    _fields_ = [
        ("split_k", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
        ("tile_k", ctypes.c_int32), ("swap_ab", ctypes.c_int32), ("num_units", ctypes.c_int32),
        ("k_per_split", ctypes.c_int32), ("repack_a", ctypes.c_int32), ("repack_b", ctypes.c_int32),
        ("kernel", ctypes.c_int32),
        ("streamk_tiles", ctypes.c_int32), ("cluster_size", ctypes.c_int32), ("dequant_form", ctypes.c_int32),
        ("realign", ctypes.c_int32),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python layout_general_tensor_gb300/build.py` "
                          "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sig = {
        "gemm_create": (ctypes.c_int, [ctypes.POINTER(gemm_desc_t), ctypes.POINTER(P)]),
        "gemm_workspace_size": (ctypes.c_int, [P, ctypes.POINTER(ctypes.c_size_t)]),
        "gemm_query": (ctypes.c_int, [P, ctypes.POINTER(gemm_info_t)]),
        "gemm_run": (ctypes.c_int, [P, P, P, P, P, P, P, ctypes.c_size_t, P]),
        "gemm_run_static_scratch": (ctypes.c_int, [P, P, P, P, P]),
        "gemm_sync_status": (ctypes.c_int, [P, P]),
        "gemm_destroy": (ctypes.c_int, [P]),
        "gemm_splitk_auto": (ctypes.c_int32, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                              ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_double]),
        "gemm_perm_fwd": (ctypes.c_uint32, [ctypes.c_uint32] * 4),
        "gemm_perm_inv": (ctypes.c_uint32, [ctypes.c_uint32] * 4),
        "gemm_perm_device": (ctypes.c_int, [P, ctypes.c_size_t, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32,
                                            ctypes.c_int32, P, P]),
        "gemm_magic_divmod_host": (ctypes.c_int, [P, ctypes.c_size_t, ctypes.c_uint32, P, P]),
        "gemm_magic_divmod_device": (ctypes.c_int, [P, ctypes.c_size_t, ctypes.c_uint32, P, P, P]),
        "gemm_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "gemm_int4_prepack_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32]),
        "gemm_int4_prepack": (ctypes.c_int, [P, ctypes.c_int64, P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                             P, P]),
        "reduce_rows_workspace_size": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                                      ctypes.POINTER(ctypes.c_size_t)]),
        "reduce_rows_f32": (ctypes.c_int, [P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, P, P,
                                           ctypes.c_size_t, P]),
        "attn_create": (ctypes.c_int, [ctypes.POINTER(attn_desc_t), ctypes.POINTER(P)]),
        "attn_run": (ctypes.c_int, [P, P, P, P, P, P]),
        "attn_sync_status": (ctypes.c_int, [P, P]),
        "attn_destroy": (ctypes.c_int, [P]),
        "attn_rope_frequencies": (ctypes.c_int, [ctypes.POINTER(attn_rope_desc_t), P]),
        "attn_rope_create": (ctypes.c_int, [ctypes.POINTER(attn_rope_desc_t), P, ctypes.POINTER(P)]),
        "attn_rope_run": (ctypes.c_int, [P, P, I64, P, I64, P, P, P, I64, P, I64, P, I64, P]),
        "attn_rope_destroy": (ctypes.c_int, [P]),
        "attn_prompt_create": (ctypes.c_int, [ctypes.POINTER(attn_prompt_desc_t), ctypes.POINTER(P)]),
        "attn_prompt_run": (ctypes.c_int, [P, P, I64, P, I64, P, I64, P, P, I32, I64, I64, P, I64, P]),
        "attn_prompt_sync_status": (ctypes.c_int, [P, P]),
        "attn_prompt_withhold_load": (ctypes.c_int, [P]),
        "attn_prompt_destroy": (ctypes.c_int, [P]),
        "attn_cache_write": (ctypes.c_int, [ctypes.POINTER(attn_cache_t), P, I64, P, I64, P, I64, I32, P]),
        "attn_cache_read": (ctypes.c_int, [ctypes.POINTER(attn_cache_t), P, I64, P, I64, P, I64, I32, P]),
        "attn_cache_attend_workspace_size": (ctypes.c_int, [I32, I32, I32, I32, ctypes.POINTER(ctypes.c_size_t)]),
        "attn_cache_attend": (ctypes.c_int, [ctypes.POINTER(attn_cache_t), P, I64, I32, P, I64, I32, P, I32,
                                             ctypes.c_float, I32, P, I64, P, ctypes.c_size_t, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()


class GemmError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__(f"{what}: {gemm_status_string(status)} ({status})")


def _check(status, what):
    if status != GEMM_OK:
        raise GemmError(status, what)


# ------------------------------------------------------------- thin wrappers

def gemm_status_string(status: int) -> str:
    return _lib.gemm_status_string(int(status)).decode()


def gemm_create(desc: gemm_desc_t) -> int:
    h = ctypes.c_void_p()
    _check(_lib.gemm_create(ctypes.byref(desc), ctypes.byref(h)), "gemm_create")
    return h.value


def gemm_create_status(desc: gemm_desc_t):
    """gemm_create returning (status, handle or None) without raising."""
    h = ctypes.c_void_p()
    st = _lib.gemm_create(ctypes.byref(desc), ctypes.byref(h))
    return st, h.value


def gemm_workspace_size(plan: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.gemm_workspace_size(plan, ctypes.byref(n)), "gemm_workspace_size")
    return n.value


def gemm_query(plan: int) -> gemm_info_t:
    info = gemm_info_t()
    _check(_lib.gemm_query(plan, ctypes.byref(info)), "gemm_query")
    return info


def gemm_run(plan: int, A: int, B: int, C: int, scales: int = 0, zeros: int = 0, workspace: int = 0,
             workspace_bytes: int = 0, stream: int = 0) -> int:
    """Raw entry point: integer device addresses; returns the status code."""
    return _lib.gemm_run(plan, A or None, B or None, C or None, scales or None, zeros or None, workspace or None,
                         workspace_bytes, stream or None)


def gemm_run_static_scratch(plan: int, A: int, B: int, C: int, stream: int = 0) -> int:
    """Run `plan` using the library's fixed device scratch instead of a
    caller workspace (for callers that cannot allocate device memory when
    they run the GEMM).  Integer device addresses; returns the status."""
    return _lib.gemm_run_static_scratch(plan, A or None, B or None, C or None, stream or None)


def gemm_sync_status(plan: int, stream: int = 0) -> int:
    return _lib.gemm_sync_status(plan, stream or None)


def gemm_destroy(plan: int) -> None:
    _check(_lib.gemm_destroy(plan), "gemm_destroy")


def gemm_splitk_auto(M, N, K, block_m=128, block_n=128, block_k=64, num_sms=148, threshold=0.05) -> int:
    return _lib.gemm_splitk_auto(M, N, K, block_m, block_n, block_k, num_sms, threshold)


def gemm_int4_prepack_bytes(N: int, K: int, group_size: int = 128) -> int:
    """Bytes of the pre-packed int4 weight buffer (0: shape not taken)."""
    return _lib.gemm_int4_prepack_bytes(N, K, group_size)


def gemm_int4_prepack(B: int, ldb: int, scales: int, N: int, K: int, group_size: int, out: int,
                      stream: int = 0) -> int:
    """Raw entry point: device addresses of the plain int4 weights, their fp16
    scales and the output buffer; returns the status."""
    return _lib.gemm_int4_prepack(B or None, ldb, scales or None, N, K, group_size, out or None, stream or None)


def gemm_perm_fwd(index, count, block, stride) -> int:
    return _lib.gemm_perm_fwd(index, count, block, stride)


def gemm_perm_inv(index, count, block, stride) -> int:
    return _lib.gemm_perm_inv(index, count, block, stride)


def gemm_perm_device(in_ptr, n, count, block, stride, inverse, out_ptr, stream=0) -> int:
    """Raw entry point: device addresses of uint32 arrays; returns the status."""
    return _lib.gemm_perm_device(in_ptr or None, n, count, block, stride, int(inverse), out_ptr or None,
                                 stream or None)


def gemm_magic_divmod_host(n_array, divisor):
    """n_array: numpy uint32 array (C-contiguous).  Returns (q, r) arrays."""
    import numpy as np
    n = np.ascontiguousarray(n_array, dtype=np.uint32)
    q = np.empty_like(n)
    r = np.empty_like(n)
    _check(_lib.gemm_magic_divmod_host(n.ctypes.data, n.size, divisor, q.ctypes.data, r.ctypes.data),
           "gemm_magic_divmod_host")
    return q, r


def gemm_magic_divmod_device(n_ptr, count, divisor, q_ptr, r_ptr, stream=0) -> int:
    return _lib.gemm_magic_divmod_device(n_ptr, count, divisor, q_ptr, r_ptr, stream or None)


def reduce_rows_workspace_size(rows: int, cols: int, num_sms: int = 0) -> int:
    n = ctypes.c_size_t()
    _check(_lib.reduce_rows_workspace_size(rows, cols, num_sms, ctypes.byref(n)), "reduce_rows_workspace_size")
    return n.value


def reduce_rows_f32(x: int, rows: int, cols: int, ldx: int, out: int, workspace: int = 0, workspace_bytes: int = 0,
                    stream: int = 0) -> int:
    """Raw entry point: integer device addresses; returns the status code."""
    return _lib.reduce_rows_f32(x or None, rows, cols, ldx, out or None, workspace or None, workspace_bytes,
                                stream or None)


def _require_device(what, **tensors):
    """Every given tensor must live in CUDA device memory: a host address
    handed to a kernel (or encoded into a tensor map) would fault the GPU
    instead of returning an error."""
    for name, t in tensors.items():
        if t is not None and not getattr(t, "is_cuda", False):
            raise ValueError(f"{what}: {name} must be a CUDA tensor")


class RowReduce:
    """out[r] = sum of row r of an fp32 matrix, with its (zero-filled) device
    workspace.  Marshalling only: passes device addresses and the current
    torch stream to reduce_rows_f32."""

    def __init__(self, rows: int, cols: int, device=None):
        import torch
        self.rows, self.cols = rows, cols
        self.ws_bytes = reduce_rows_workspace_size(rows, cols, 0)
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        self.workspace = torch.zeros(max(self.ws_bytes, 1), dtype=torch.uint8, device=dev)

    def run(self, x, out, ldx: int = 0, stream=None):
        import torch
        _require_device("RowReduce.run", x=x, out=out)
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream
        st = reduce_rows_f32(x.data_ptr(), self.rows, self.cols, ldx, out.data_ptr(),
                             self.workspace.data_ptr() if self.ws_bytes else 0, self.ws_bytes, s)
        _check(st, "reduce_rows_f32")


def make_desc(M, N, K, a_layout=GEMM_K_CONTIG, b_layout=GEMM_K_CONTIG, a_dtype=GEMM_BF16, b_dtype=None,
              c_dtype=None, lda=0, ldb=0, ldc=0, split_k=1, group_size=0, num_sms=0, flags=0) -> gemm_desc_t:
    b_dtype = a_dtype if b_dtype is None else b_dtype
    c_dtype = a_dtype if c_dtype is None else c_dtype
    return gemm_desc_t(M, N, K, a_layout, b_layout, lda, ldb, ldc, a_dtype, b_dtype, c_dtype, split_k,
                       group_size, num_sms, flags)


class Gemm:
    """A plan plus its (zero-filled) device workspace, run on torch tensors.

    Marshalling only: passes the tensors' device addresses and the current
    torch stream to gemm_run."""

    def __init__(self, desc: gemm_desc_t, device=None):
        import torch
        self.desc = desc
        self.plan = gemm_create(desc)
        self.info = gemm_query(self.plan)
        self.ws_bytes = gemm_workspace_size(self.plan)
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        self.workspace = torch.zeros(max(self.ws_bytes, 1), dtype=torch.uint8, device=dev)

    def run(self, A, B, C, scales=None, zeros=None, stream=None, workspace=None, workspace_bytes=None):
        import torch
        ws = self.workspace if workspace is None else workspace
        wsb = self.ws_bytes if workspace_bytes is None else workspace_bytes
        _require_device("Gemm.run", A=A, B=B, C=C, scales=scales, zeros=zeros, workspace=ws if wsb else None)
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream
        st = gemm_run(self.plan, A.data_ptr(), B.data_ptr(), C.data_ptr(),
                      scales.data_ptr() if scales is not None else 0,
                      zeros.data_ptr() if zeros is not None else 0,
                      ws.data_ptr() if wsb else 0, wsb, s)
        _check(st, "gemm_run")

    def sync_status(self, stream=None) -> int:
        import torch
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream
        return gemm_sync_status(self.plan, s)

    def close(self):
        if self.plan:
            gemm_destroy(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def int4_prepack(B, scales, N, K, group_size=128, ldb=0, stream=None):
    """Pre-pack int4 weights (device uint8 tensor, N rows of ldb bytes) and
    their fp16 scales for GEMM_FLAG_INT4_PREPACKED; returns the packed device
    uint8 tensor."""
    import torch
    _require_device("int4_prepack", B=B, scales=scales)
    nbytes = gemm_int4_prepack_bytes(N, K, group_size)
    if nbytes == 0:
        raise GemmError(GEMM_ERR_INVALID_ARG, "gemm_int4_prepack_bytes")
    out = torch.empty(nbytes, dtype=torch.uint8, device=B.device)
    s = torch.cuda.current_stream().cuda_stream if stream is None else stream
    _check(gemm_int4_prepack(B.data_ptr(), ldb, scales.data_ptr(), N, K, group_size, out.data_ptr(), s),
           "gemm_int4_prepack")
    return out


def attn_create_status(desc: attn_desc_t):
    """attn_create returning (status, handle or None) without raising."""
    h = ctypes.c_void_p()
    st = _lib.attn_create(ctypes.byref(desc), ctypes.byref(h))
    return st, h.value


def attn_run(plan: int, Q: int, K: int, V: int, O: int, stream: int = 0) -> int:
    """Raw entry point: integer device addresses; returns the status code."""
    return _lib.attn_run(plan, Q or None, K or None, V or None, O or None, stream or None)


class Attention:
    """A fused-attention plan run on torch tensors laid out [head][row][d]
    (marshalling only: the tensors' device addresses and the current torch
    stream go to attn_run)."""

    def __init__(self, heads, seq_q, seq_k, head_dim, dtype=GEMM_BF16, scale=0.0):
        self.desc = attn_desc_t(heads, seq_q, seq_k, head_dim, dtype, scale)
        st, h = attn_create_status(self.desc)
        _check(st, "attn_create")
        self.plan = h

    def run(self, Q, K, V, O, stream=None):
        import torch
        _require_device("Attention.run", Q=Q, K=K, V=V, O=O)
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream
        _check(attn_run(self.plan, Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), s), "attn_run")

    def sync_status(self, stream=None) -> int:
        import torch
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream
        return _lib.attn_sync_status(self.plan, s or None)

    def close(self):
        if self.plan:
            _lib.attn_destroy(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_torch = None
_binding = None


def _with_torch():
    """torch and the binding's part in C (csrc/binding.c), which goes by
    torch's types; both at the first use, the rest does without."""
    global _torch, _binding
    import importlib.util

    import torch
    if not os.path.exists(_BINDING_PATH):
        raise ImportError(f"{_BINDING_PATH} is missing: build it with `python layout_general_tensor_gb300/build.py`, "
                          "with a C compiler and Python's headers (there is no other way to the serving operators)")
    loader = importlib.machinery.ExtensionFileLoader("_binding", _BINDING_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_binding", loader))
    loader.exec_module(module)
    # (the plain way to the current stream costs 3.5 us a call on the host)
    raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)
    module.setup(*(ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value for name in
                   ("attn_rope_run", "attn_prompt_run", "attn_cache_write", "attn_cache_read", "attn_cache_attend")),
                 getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device, raw_stream, torch.int32,
                 torch.float16, torch.bfloat16)
    _torch, _binding = torch, module
    return torch


def _torch_dtype(dtype):
    torch = _torch or _with_torch()
    return torch.bfloat16 if dtype == GEMM_BF16 else torch.float16


def _refuse(what, status, *checks, kept=()):
    """Raise for a call's status; at -1 the binding refused a tensor: find it
    among checks of (name, tensor, shape, torch type, whether its rows may be
    strided), or in `kept`, pairs of (name, device) of what the object holds."""
    if status != -1:
        _check(status, what)
    for name, t, shape, dtype, rows in checks:
        if not getattr(t, "is_cuda", False):
            raise ValueError(f"{what}: {name} must be a CUDA tensor")
        kept = (*kept, (name, t.get_device()))
        if t.dtype is not dtype or tuple(t.shape) != tuple(shape):
            raise ValueError(f"{what}: {name} must be {list(shape)} of {dtype}, got {list(t.shape)} of {t.dtype}")
        if not rows and not t.is_contiguous():
            raise ValueError(f"{what}: {name} must be contiguous")
    for name, device in kept:
        if device != _torch.cuda.current_device():
            raise ValueError(f"{what}: {name} is on cuda:{device}, the current device is cuda:{_torch.cuda.current_device()}")
    raise ValueError(f"{what}: within a row the values of a tensor must be contiguous, and rows must not overlap")


def attn_rope_frequencies(desc: attn_rope_desc_t):
    """The frequencies (radians a position) `desc` stands for, as a list."""
    out = (ctypes.c_double * max(desc.rot_dim // 2, 1))()
    _check(_lib.attn_rope_frequencies(ctypes.byref(desc), out), "attn_rope_frequencies")
    return list(out)[: desc.rot_dim // 2]


def attn_rope_create_status(desc: attn_rope_desc_t, frequencies=None):
    """attn_rope_create returning (status, handle or None) without raising."""
    h = ctypes.c_void_p()
    f = None if frequencies is None else (ctypes.c_double * max(len(frequencies), 1))(*frequencies)
    return _lib.attn_rope_create(ctypes.byref(desc), f, ctypes.byref(h)), h.value


class QKNormRope:
    """The RMS norm of every query and key head and its rotation by position,
    in one pass over [token][head][head_dim] tensors, which may be slices of
    one projection's output (include/attn_rope.h).  Without weights there is
    no norm.  `frequencies` (rot_dim / 2 radians a position) takes the place
    of base, factor, context, low_turns and high_turns.  The tensors of a call
    are on the current device."""

    def __init__(self, q_heads, k_heads, head_dim, rot_dim=None, layout=ATTN_ROPE_HALF, dtype=GEMM_BF16, eps=1e-6,
                 base=10000.0, factor=1.0, context=0.0, low_turns=0.0, high_turns=0.0, magnitude=1.0,
                 frequencies=None):
        rot_dim = head_dim if rot_dim is None else rot_dim
        self.plan = None
        self.desc = attn_rope_desc_t(q_heads, k_heads, head_dim, rot_dim, layout, dtype, eps, magnitude, base, factor,
                                     context, low_turns, high_turns)
        if frequencies is not None and len(frequencies) != rot_dim // 2:
            raise ValueError(f"QKNormRope: {rot_dim // 2} frequencies are wanted, got {len(frequencies)}")
        st, h = attn_rope_create_status(self.desc, frequencies)
        _check(st, "attn_rope_create")
        self.plan = h
        self.dtype = _torch_dtype(dtype)
        self.handle = (h, self.dtype, q_heads, k_heads, head_dim)

    def run(self, q, k, positions, q_out, k_out, q_weight=None, k_weight=None, stream=None):
        """q_out, k_out: may be q and k themselves.  positions: int32."""
        st = _binding.rope(self.handle, q, k, positions, q_out, k_out, q_weight, k_weight, stream)
        if st:
            d, dt, n = self.desc, self.dtype, len(q)
            qs, ks, ws = (n, d.q_heads, d.head_dim), (n, d.k_heads, d.head_dim), (d.head_dim,)
            _refuse("attn_rope_run", st, ("q", q, qs, dt, True), ("k", k, ks, dt, True),
                    ("positions", positions, (n,), _torch.int32, False), ("q_out", q_out, qs, dt, True),
                    ("k_out", k_out, ks, dt, True),
                    *((name, w, ws, dt, False) for name, w in (("q_weight", q_weight), ("k_weight", k_weight)) if w is not None))

    def close(self):
        if self.plan:
            _lib.attn_rope_destroy(self.plan)
            self.plan, self.handle = None, (0, *self.handle[1:])

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def attn_prompt_create_status(desc: attn_prompt_desc_t):
    """attn_prompt_create returning (status, handle or None) without raising."""
    h = ctypes.c_void_p()
    return _lib.attn_prompt_create(ctypes.byref(desc), ctypes.byref(h)), h.value


class PromptAttention:
    """Attention over packed sequences of different lengths, causal or not,
    with grouped heads (include/attn_prompt.h), on [row][head][head_dim]
    tensors and cumulative lengths (batch + 1 int32 on the device).  The tensors
    of a call are on the current device, the one the object was made on.  A graph
    needs the object that it was captured from (its status word)."""

    def __init__(self, q_heads, k_heads, head_dim, dtype=GEMM_BF16, causal=True, scale=0.0):
        self.plan = None
        self.desc = attn_prompt_desc_t(q_heads, k_heads, head_dim, dtype, int(causal), scale)
        st, h = attn_prompt_create_status(self.desc)
        _check(st, "attn_prompt_create")
        self.plan = h
        self.dtype = _torch_dtype(dtype)
        self.handle = (h, self.dtype, q_heads, k_heads, head_dim)

    def run(self, q, k, v, cu_q, cu_k, out, stream=None):
        st = _binding.prompt(self.handle, q, k, v, cu_q, cu_k, out, stream)
        if st:
            d, dt, n, nk, cus = self.desc, self.dtype, len(q), len(k), len(cu_q)
            qs, ks = (n, d.q_heads, d.head_dim), (nk, d.k_heads, d.head_dim)
            if st == -1 and cus < 1:
                raise ValueError("attn_prompt_run: cu_q and cu_k hold batch + 1 values")
            _refuse("attn_prompt_run", st, ("q", q, qs, dt, True), ("k", k, ks, dt, True), ("v", v, ks, dt, True),
                    ("cu_q", cu_q, (cus,), _torch.int32, False), ("cu_k", cu_k, (cus,), _torch.int32, False),
                    ("out", out, qs, dt, True))

    def sync_status(self, stream=None) -> int:
        torch = _torch or _with_torch()
        return _lib.attn_prompt_sync_status(self.plan, torch.cuda.current_stream().cuda_stream if stream is None else stream)

    def close(self):
        if self.plan:
            _lib.attn_prompt_destroy(self.plan)
            self.plan, self.handle = None, (0, *self.handle[1:])

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KVCache:
    """A paged cache of keys and values in 8 bits (include/attn_cache.h), on
    four uint8 tensors: codes [pages][k_heads][page_size][head_dim] and
    exponents [pages][k_heads][page_size].  They and the tensors of a call are
    on the current device."""

    def __init__(self, k, v, k_exp, v_exp):
        torch = _torch or _with_torch()
        for name, t in (("k", k), ("v", v), ("k_exp", k_exp), ("v_exp", v_exp)):
            if not getattr(t, "is_cuda", False) or t.dtype != torch.uint8 or not t.is_contiguous():
                raise ValueError(f"KVCache: {name} must be a contiguous CUDA tensor of uint8")
            if t.get_device() != k.get_device():
                raise ValueError(f"KVCache: {name} is on another device than k")
        if k.dim() != 4 or v.shape != k.shape or k_exp.shape != k.shape[:3] or v_exp.shape != k.shape[:3]:
            raise ValueError("KVCache: codes are [pages][k_heads][page_size][head_dim], exponents one dimension less")
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp
        self.pages, self.k_heads, self.page_size, self.head_dim = k.shape
        self.c = attn_cache_t(k.data_ptr(), v.data_ptr(), k_exp.data_ptr(), v_exp.data_ptr(), self.pages,
                              self.page_size, self.k_heads, self.head_dim)
        self._ref, self.address = ctypes.byref(self.c), ctypes.addressof(self.c)
        self.handle = (self.address, self.k_heads, self.head_dim, k.get_device())

    @classmethod
    def empty(cls, pages, page_size, k_heads, head_dim, device="cuda"):
        import torch
        made = [torch.zeros(pages, k_heads, page_size, head_dim, dtype=torch.uint8, device=device) for _ in range(2)]
        made += [torch.zeros(pages, k_heads, page_size, dtype=torch.uint8, device=device) for _ in range(2)]
        return cls(*made)

    def write(self, k, v, slots, stream=None):
        """Quantise [token][k_heads][head_dim] keys and values into their slots (int32, distinct within a call;
        negative: left out, which is the way to pad)."""
        st = _binding.cache_write(self.handle, k, v, slots, stream)
        if st:
            self._refuse("attn_cache_write", st, k, v, slots)

    def read(self, slots, k, v, stream=None):
        """The values of the slots into [token][k_heads][head_dim] tensors (zeros for a negative slot)."""
        st = _binding.cache_read(self.handle, k, v, slots, stream)
        if st:
            self._refuse("attn_cache_read", st, k, v, slots)

    def _refuse(self, what, st, k, v, slots):
        if st == -1 and k.dtype not in (_torch.float16, _torch.bfloat16):
            raise ValueError(f"{what}: k and v must be float16 or bfloat16, got {k.dtype}")
        n = len(k)
        shape = (n, self.k_heads, self.head_dim)
        _refuse(what, st, ("k", k, shape, k.dtype, True), ("v", v, shape, k.dtype, True),
                ("slots", slots, (n,), _torch.int32, False), kept=(("the cache", self.handle[3]),))


class CacheAttention:
    """Attention of one query a sequence over a KVCache (include/attn_cache.h),
    with its (zero-filled) device workspace for `batch` sequences.  A larger batch
    waits for the device and makes a larger one; the one before is kept as long as
    the object is, since a captured graph goes on using it.  While a graph is being
    captured there is no waiting, so a larger batch is refused: make the object for
    the largest one.  Runs that may be under way at the same time need objects of
    their own, and a graph needs the object that it was captured from.  The tensors
    of a call and the cache are on the current device, the one the object was made
    on."""

    def __init__(self, q_heads, k_heads, head_dim, page_size, dtype=GEMM_BF16, scale=0.0, batch=64):
        self.q_heads, self.k_heads, self.head_dim, self.page_size = q_heads, k_heads, head_dim, page_size
        self.dtype, self.scale, self.code = _torch_dtype(dtype), scale, dtype
        self.workspace, self.ws_bytes, self.batch, self._earlier = None, 0, 0, []
        self._grow(batch)

    def _grow(self, batch):
        torch = _torch
        n = ctypes.c_size_t()
        _check(_lib.attn_cache_attend_workspace_size(self.q_heads, self.k_heads, self.head_dim, batch,
                                                     ctypes.byref(n)), "attn_cache_attend_workspace_size")
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError(f"CacheAttention: the workspace is for {self.batch} sequences and cannot be made larger while a "
                               f"graph is being captured: make the object with batch={batch} before")
        # (the old one may be in use and the new one is used on any stream)
        torch.cuda.synchronize()
        if self.workspace is not None:
            self._earlier.append(self.workspace)
        self.workspace = torch.zeros(n.value, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        self.ws_bytes, self.batch = n.value, batch
        self.handle = (self.dtype, self.q_heads, self.k_heads, self.head_dim, self.page_size, self.code, float(self.scale),
                       self.workspace.data_ptr(), self.ws_bytes, batch, self.workspace.get_device())

    def run(self, q, cache, page_table, lengths, out, stream=None):
        """q, out: [batch][q_heads][head_dim]; page_table: [batch][pages a sequence] int32; lengths: batch int32."""
        st = _binding.attend(self.handle, cache.handle, q, page_table, lengths, out, stream)
        if st == -2:
            # (twice as many at least, up to the library's most: what is kept stays a few times the last)
            self._grow(max(len(q), min(2 * self.batch, 8192)))
            st = _binding.attend(self.handle, cache.handle, q, page_table, lengths, out, stream)
        if st:
            what, n, dt = "attn_cache_attend", len(q), self.dtype
            if st == -1 and (cache.k_heads, cache.head_dim, cache.page_size) != (self.k_heads, self.head_dim, self.page_size):
                raise ValueError(f"{what}: the cache has another shape than this was made for")
            shape = (n, self.q_heads, self.head_dim)
            _refuse(what, st, ("q", q, shape, dt, True), ("page_table", page_table, (n, page_table.shape[-1]), _torch.int32, True),
                    ("lengths", lengths, (n,), _torch.int32, False), ("out", out, shape, dt, True),
                    kept=(("the workspace", self.handle[10]), ("the cache", cache.handle[3])))
