"""ctypes binding of libqkgemv.so (declared in include/qkgemv.h).

Argument marshalling only: every step of the GEMV runs in the library's HIP
kernels.  The raw entry points keep the C names and take integer device
addresses; ``gemv`` / ``dequant`` accept torch tensors and pass their data
pointers and the current HIP stream.  If the library is not built, every call
raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqkgemv.so")

Q4_K, Q5_K, Q6_K, IQ4_XS = 12, 13, 14, 23
QK_OK, QK_EINVAL_TYPE, QK_EINVAL_SHAPE, QK_EINVAL_PTR, QK_ELAUNCH, QK_EINVAL_FLAGS = 0, -1, -2, -3, -4, -5
MAX_NCOLS = 32
MAX_BATCH = 16
PLANAR = 0x100  # QK_PLANAR: layout flag OR'ed into a type
Y_F16 = 0x1  # QK_Y_F16: epilogue flag, y stored as fp16

EXPORTS = ("qk_gemv", "qk_gemv_ex", "qk_gemv_swiglu", "qk_gemv_batch", "qk_dequant", "qk_repack",
           "qk_block_bytes", "qk_row_bytes", "qk_strerror", "qk_version",
           "qk_chain_plan_bytes", "qk_chain_plan", "qk_chain_workspace_bytes", "qk_gemv_chain",
           "qk_gemv_chain_noalloc",
           "qk_norm_rope", "qk_kv_page_bytes", "qk_kv_append", "qk_kv_read", "qk_kv_attn_workspace_bytes",
           "qk_kv_attn")
CHAIN_TIMEOUT = 0x1  # QK_CHAIN_TIMEOUT: bit of the chain workspace's first word
CHAIN_NOALLOC_MAX_STEPS = 4094  # QK_CHAIN_NOALLOC_MAX_STEPS


class qk_gemv_item(ctypes.Structure):
    """struct qk_gemv_item of include/qkgemv.h."""
    _fields_ = [("type", ctypes.c_int), ("W", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class qk_chain_entry(ctypes.Structure):
    """struct qk_chain_entry of include/qkgemv.h."""
    _fields_ = [("type", ctypes.c_int), ("flags", ctypes.c_int), ("W", ctypes.c_void_p), ("W2", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class qk_heads(ctypes.Structure):
    """struct qk_heads of include/qkgemv.h."""
    _fields_ = [("p", ctypes.c_void_p), ("row", ctypes.c_int64), ("head", ctypes.c_int64), ("elem", ctypes.c_int64),
                ("f16", ctypes.c_int)]


class qk_rope(ctypes.Structure):
    """struct qk_rope of include/qkgemv.h."""
    _fields_ = [("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("eps", ctypes.c_float), ("rot_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int)]


class qk_kv_cache(ctypes.Structure):
    """struct qk_kv_cache of include/qkgemv.h."""
    _fields_ = [("pool", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int)]


class qk_kv_seqs(ctypes.Structure):
    """struct qk_kv_seqs of include/qkgemv.h."""
    _fields_ = [("rows", ctypes.c_int), ("nseq", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("pages", ctypes.c_void_p)]


class QKError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {qk_strerror(code)} (code {code})")
        self.code = code


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libqkgemv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run quant_dequant_gemv_amd/build.py "
                          "(or __graft_entry__.build()) first")
    lib = ctypes.CDLL(path)
    P, i64, c_int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.qk_gemv.argtypes = [c_int, P, P, P, i64, i64, c_int, P]
    lib.qk_gemv.restype = c_int
    lib.qk_gemv_ex.argtypes = [c_int, P, P, P, i64, i64, c_int, P, c_int, P]
    lib.qk_gemv_ex.restype = c_int
    lib.qk_gemv_swiglu.argtypes = [c_int, P, P, P, P, i64, i64, c_int, c_int, P]
    lib.qk_gemv_swiglu.restype = c_int
    lib.qk_gemv_batch.argtypes = [ctypes.POINTER(qk_gemv_item), c_int, P]
    lib.qk_gemv_batch.restype = c_int
    lib.qk_dequant.argtypes = [c_int, P, P, i64, i64, P]
    lib.qk_dequant.restype = c_int
    lib.qk_repack.argtypes = [c_int, P, P, i64, i64, P]
    lib.qk_repack.restype = c_int
    lib.qk_block_bytes.argtypes = [c_int]
    lib.qk_block_bytes.restype = c_int
    lib.qk_row_bytes.argtypes = [c_int, i64]
    lib.qk_row_bytes.restype = i64
    lib.qk_strerror.argtypes = [c_int]
    lib.qk_strerror.restype = ctypes.c_char_p
    lib.qk_version.argtypes = []
    lib.qk_version.restype = ctypes.c_char_p
    lib.qk_chain_plan_bytes.argtypes = [c_int, c_int]
    lib.qk_chain_plan_bytes.restype = i64
    lib.qk_chain_plan.argtypes = [ctypes.POINTER(qk_chain_entry), c_int, ctypes.POINTER(c_int), c_int, P, i64]
    lib.qk_chain_plan.restype = c_int
    lib.qk_chain_workspace_bytes.argtypes = [c_int]
    lib.qk_chain_workspace_bytes.restype = i64
    lib.qk_gemv_chain.argtypes = [P, P, P, i64, i64, P]
    lib.qk_gemv_chain.restype = c_int
    lib.qk_gemv_chain_noalloc.argtypes = [P, P, P, i64, P]
    lib.qk_gemv_chain_noalloc.restype = c_int
    H, R = ctypes.POINTER(qk_heads), ctypes.POINTER(qk_rope)
    C, S = ctypes.POINTER(qk_kv_cache), ctypes.POINTER(qk_kv_seqs)
    lib.qk_norm_rope.argtypes = [R, c_int, c_int, c_int, H, H, c_int, H, H, P]
    lib.qk_norm_rope.restype = c_int
    lib.qk_kv_page_bytes.argtypes = [c_int, c_int, c_int]
    lib.qk_kv_page_bytes.restype = i64
    lib.qk_kv_append.argtypes = [C, S, R, H, H, c_int, H, H, P]
    lib.qk_kv_append.restype = c_int
    lib.qk_kv_read.argtypes = [C, S, H, H, P]
    lib.qk_kv_read.restype = c_int
    lib.qk_kv_attn_workspace_bytes.argtypes = [C, S, c_int]
    lib.qk_kv_attn_workspace_bytes.restype = i64
    lib.qk_kv_attn.argtypes = [C, S, c_int, H, H, ctypes.c_float, c_int, P, i64, P]
    lib.qk_kv_attn.restype = c_int
    _lib = lib
    return lib


# ---------------------------------------------------------------- raw C names

def qk_gemv(qtype: int, W: int, x: int, y: int, N: int, K: int, ncols: int, stream: int = 0) -> int:
    return load_library().qk_gemv(qtype, W, x, y, N, K, ncols, stream)


def qk_gemv_ex(qtype: int, W: int, x: int, y: int, N: int, K: int, ncols: int, residual, flags: int,
               stream: int = 0) -> int:
    return load_library().qk_gemv_ex(qtype, W, x, y, N, K, ncols, residual, flags, stream)


def qk_gemv_swiglu(qtype: int, Wg: int, Wu: int, x: int, y: int, N: int, K: int, ncols: int, flags: int,
                   stream: int = 0) -> int:
    return load_library().qk_gemv_swiglu(qtype, Wg, Wu, x, y, N, K, ncols, flags, stream)


def qk_gemv_batch(items, stream: int = 0) -> int:
    """items: sequence of (type, W, x, y, N, K) with integer device addresses."""
    arr = (qk_gemv_item * max(1, len(items)))(*[qk_gemv_item(*it) for it in items])
    return load_library().qk_gemv_batch(arr, len(items), stream)


def qk_chain_plan_bytes(nsteps: int, nentries: int) -> int:
    return load_library().qk_chain_plan_bytes(nsteps, nentries)


def qk_chain_plan(entries, step_sizes, plan) -> int:
    """entries: sequence of qk_chain_entry (or tuples of its fields);
    step_sizes: ints; plan: a writable host buffer (numpy uint8 array)."""
    arr = (qk_chain_entry * max(1, len(entries)))(*[e if isinstance(e, qk_chain_entry) else qk_chain_entry(*e)
                                                     for e in entries])
    sizes = (ctypes.c_int * max(1, len(step_sizes)))(*step_sizes)
    return load_library().qk_chain_plan(arr, len(entries), sizes, len(step_sizes),
                                        ctypes.c_void_p(plan.ctypes.data), int(plan.nbytes))


def qk_chain_workspace_bytes(nsteps: int) -> int:
    return load_library().qk_chain_workspace_bytes(nsteps)


def qk_gemv_chain(plan, plan_dev: int, workspace: int, workspace_bytes: int, timeout_us: int = 0,
                  stream: int = 0) -> int:
    """plan: the host plan (numpy uint8 array)."""
    return load_library().qk_gemv_chain(ctypes.c_void_p(plan.ctypes.data), plan_dev, workspace, workspace_bytes,
                                        timeout_us, stream)


def qk_gemv_chain_noalloc(plan, plan_dev: int, status: int = 0, timeout_us: int = 0, stream: int = 0) -> int:
    """plan: the host plan (numpy uint8 array); status: 0 or a device word."""
    return load_library().qk_gemv_chain_noalloc(ctypes.c_void_p(plan.ctypes.data), plan_dev, status, timeout_us,
                                                stream)


def qk_dequant(qtype: int, W: int, out: int, N: int, K: int, stream: int = 0) -> int:
    return load_library().qk_dequant(qtype, W, out, N, K, stream)


def qk_repack(qtype: int, W: int, Wp: int, N: int, K: int, stream: int = 0) -> int:
    return load_library().qk_repack(qtype, W, Wp, N, K, stream)


def qk_block_bytes(qtype: int) -> int:
    return load_library().qk_block_bytes(qtype)


def qk_row_bytes(qtype: int, K: int) -> int:
    return load_library().qk_row_bytes(qtype, K)


def qk_strerror(code: int) -> str:
    return load_library().qk_strerror(code).decode()


def qk_version() -> str:
    return load_library().qk_version().decode()


def qk_norm_rope(rope, rows: int, head_dim: int, n_heads: int, q, q_out, n_kv_heads: int, k, k_out,
                 stream: int = 0) -> int:
    """rope: a qk_rope; q, q_out, k, k_out: qk_heads or None."""
    return load_library().qk_norm_rope(rope, rows, head_dim, n_heads, q, q_out, n_kv_heads, k, k_out, stream)


def qk_kv_page_bytes(head_dim: int, n_kv_heads: int, page_size: int) -> int:
    return load_library().qk_kv_page_bytes(head_dim, n_kv_heads, page_size)


def qk_kv_append(cache, seqs, rope, k, v, n_heads: int, q, q_out, stream: int = 0) -> int:
    """cache: qk_kv_cache; seqs: qk_kv_seqs; rope: qk_rope or None; k, v, q, q_out: qk_heads (q, q_out or None)."""
    return load_library().qk_kv_append(cache, seqs, rope, k, v, n_heads, q, q_out, stream)


def qk_kv_read(cache, seqs, k_out, v_out, stream: int = 0) -> int:
    return load_library().qk_kv_read(cache, seqs, k_out, v_out, stream)


def qk_kv_attn_workspace_bytes(cache, seqs, n_heads: int) -> int:
    return load_library().qk_kv_attn_workspace_bytes(cache, seqs, n_heads)


def qk_kv_attn(cache, seqs, n_heads: int, q, out, scale: float, window: int, workspace, workspace_bytes: int,
               stream: int = 0) -> int:
    return load_library().qk_kv_attn(cache, seqs, n_heads, q, out, scale, window, workspace, workspace_bytes, stream)


# ---------------------------------------------------------------- torch helpers
# The C ABI cannot see buffer lengths, so these helpers check every tensor
# before anything is enqueued: dtype, contiguity, size against N, K and ncols,
# and that all of them sit on one CUDA device.  (A wrong size or a host tensor
# passed on would make a kernel read or write out of bounds.)  Type and shape
# arguments themselves are checked by the library, which returns its error
# code before launching anything.

def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _need(t, name, dtype, numel=None, min_numel=None):
    """Check one tensor argument (sizes before the device, so the checks run
    without a GPU too)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, has {t.numel()}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} must have at least {min_numel} elements, has {t.numel()}")


def _same_cuda_device(**tensors):
    devs = {t.device for t in tensors.values() if t is not None}
    for name, t in tensors.items():
        if t is not None and t.device.type != "cuda":
            raise ValueError(f"{name} must be a CUDA (HIP) device tensor, is on {t.device}")
    if len(devs) > 1:
        raise ValueError(f"all tensors must be on one device, got {sorted(str(d) for d in devs)}")


def _weights(qtype, W, N, K, name="W"):
    """W: uint8, at least N rows of qk_row_bytes(qtype, K) bytes (skipped when
    the library would reject the type or shape itself)."""
    import torch
    rb = qk_row_bytes(qtype, K) if isinstance(qtype, int) else -1
    _need(W, name, torch.uint8, min_numel=N * rb if (rb > 0 and N >= 1) else None)


def _activations(x, K):
    """x: float16 [K'] or [K', ncols] with K' >= K (the kernels read the first
    K rows: a longer buffer is a valid input); returns ncols."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch tensor")
    if x.dim() not in (1, 2) or x.shape[0] < K:
        raise ValueError(f"x must have shape [K] or [K, ncols] with at least K = {K} rows, got {tuple(x.shape)}")
    ncols = 1 if x.dim() == 1 else int(x.shape[1])
    _need(x, "x", torch.float16, min_numel=K * ncols)
    return ncols


def gemv(qtype: int, W, x, N: int, K: int, out=None, stream=None):
    """y = dequant(W) @ x on the GPU.  W: uint8 device tensor of N rows of
    superblocks; x: float16 device tensor [K] or [K, ncols]; returns float32
    [N, ncols] (or writes ``out``, N*ncols float32 elements)."""
    import torch
    _weights(qtype, W, N, K)
    ncols = _activations(x, K)
    if out is None:
        out = torch.empty((max(N, 0), ncols), dtype=torch.float32, device=x.device)
    _need(out, "out", torch.float32, numel=N * ncols)
    _same_cuda_device(W=W, x=x, out=out)
    rc = qk_gemv(qtype, W.data_ptr(), x.data_ptr(), out.data_ptr(), N, K, ncols, _stream_handle(stream))
    if rc != QK_OK:
        raise QKError(rc, "qk_gemv")
    return out


def _check_out(x, out, f16, N, ncols):
    import torch
    dt = torch.float16 if f16 else torch.float32
    if out is None:
        out = torch.empty((max(N, 0), ncols), dtype=dt, device=x.device)
    _need(out, "out", dt, numel=N * ncols)
    return out


def gemv_ex(qtype: int, W, x, N: int, K: int, residual=None, f16: bool = False, out=None, stream=None):
    """y = residual + dequant(W) @ x, stored as float32 (or float16 with f16).
    residual: None or a float32 device tensor of N*ncols elements (may be
    ``out`` itself for an in-place update of a float32 y)."""
    import torch
    _weights(qtype, W, N, K)
    ncols = _activations(x, K)
    out = _check_out(x, out, f16, N, ncols)
    if residual is not None:
        _need(residual, "residual", torch.float32, numel=N * ncols)
    _same_cuda_device(W=W, x=x, out=out, residual=residual)
    rp = residual.data_ptr() if residual is not None else None
    rc = qk_gemv_ex(qtype, W.data_ptr(), x.data_ptr(), out.data_ptr(), N, K, ncols, rp,
                    Y_F16 if f16 else 0, _stream_handle(stream))
    if rc != QK_OK:
        raise QKError(rc, "qk_gemv_ex")
    return out


def gemv_swiglu(qtype: int, Wg, Wu, x, N: int, K: int, f16: bool = False, out=None, stream=None):
    """y = silu(dequant(Wg) @ x) * (dequant(Wu) @ x) in one launch."""
    _weights(qtype, Wg, N, K, "Wg")
    _weights(qtype, Wu, N, K, "Wu")
    ncols = _activations(x, K)
    out = _check_out(x, out, f16, N, ncols)
    _same_cuda_device(Wg=Wg, Wu=Wu, x=x, out=out)
    rc = qk_gemv_swiglu(qtype, Wg.data_ptr(), Wu.data_ptr(), x.data_ptr(), out.data_ptr(), N, K, ncols,
                        Y_F16 if f16 else 0, _stream_handle(stream))
    if rc != QK_OK:
        raise QKError(rc, "qk_gemv_swiglu")
    return out


def gemv_batch(entries, stream=None):
    """Independent one-column GEMVs in one launch.  entries: sequence of
    (qtype, W, x, N, K) or (qtype, W, x, N, K, out) with torch device tensors
    (W uint8, x float16 [K], out float32 [N]); returns the list of outputs."""
    import torch
    items, outs = [], []
    for i, e in enumerate(entries):
        qtype, W, x, N, K = e[:5]
        _weights(qtype, W, N, K, f"entries[{i}].W")
        if _activations(x, K) != 1:
            raise ValueError(f"entries[{i}].x must be one column")
        out = e[5] if len(e) > 5 else torch.empty(max(N, 0), dtype=torch.float32, device=x.device)
        _need(out, f"entries[{i}].out", torch.float32, numel=N)
        items.append((qtype, W, x, out, N, K))
        outs.append(out)
    tensors = {}
    for i, (_, W, x, out, _, _) in enumerate(items):
        tensors.update({f"entries[{i}].W": W, f"entries[{i}].x": x, f"entries[{i}].out": out})
    if tensors:
        _same_cuda_device(**tensors)
    items = [(qt, W.data_ptr(), x.data_ptr(), out.data_ptr(), N, K) for qt, W, x, out, N, K in items]
    rc = qk_gemv_batch(items, _stream_handle(stream))
    if rc != QK_OK:
        raise QKError(rc, "qk_gemv_batch")
    return outs


def dequant(qtype: int, W, N: int, K: int, out=None, stream=None):
    """fp32 [N, K] dequantised weights on the GPU (``out``: N*K float32)."""
    import torch
    _weights(qtype, W, N, K)
    if out is None:
        out = torch.empty((max(N, 0), max(K, 0)), dtype=torch.float32, device=W.device)
    _need(out, "out", torch.float32, numel=N * K)
    _same_cuda_device(W=W, out=out)
    rc = qk_dequant(qtype, W.data_ptr(), out.data_ptr(), N, K, _stream_handle(stream))
    if rc != QK_OK:
        raise QKError(rc, "qk_dequant")
    return out


def repack(qtype: int, W, N: int, K: int, out=None, stream=None):
    """GGUF rows -> PLANAR rows on the GPU; returns the uint8 device tensor to
    pass with type ``qtype | PLANAR`` (``out``: at least
    N * qk_row_bytes(qtype | PLANAR, K) bytes)."""
    import torch
    _weights(qtype, W, N, K)
    prb = qk_row_bytes(qtype | PLANAR, K) if isinstance(qtype, int) and not (qtype & PLANAR) else -1
    nbytes = N * prb if (prb > 0 and N >= 1) else 0
    if out is None:
        out = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=W.device)
    _need(out, "out", torch.uint8, min_numel=nbytes or None)
    _same_cuda_device(W=W, out=out)
    rc = qk_repack(qtype, W.data_ptr(), out.data_ptr(), N, K, _stream_handle(stream))
    if rc != QK_OK:
        raise QKError(rc, "qk_repack")
    return out


class Chain:
    """A planned chain of one-column GEMV steps (qk_chain_plan / qk_gemv_chain).

    steps: list of steps; each step a list of dicts with keys qtype, W, x, y,
    N, K and optionally W2 (SwiGLU up tensor), residual (fp32, may be y) and
    f16 (y stored as fp16).  Every tensor is checked like the other helpers
    check theirs; the plan is uploaded once and the workspace allocated here,
    so run() enqueues the chain and nothing else."""

    def __init__(self, steps):
        import numpy as np
        import torch
        entries, sizes, keep = [], [], []
        for s, step in enumerate(steps):
            if not step:
                raise ValueError(f"step {s} is empty")
            sizes.append(len(step))
            for i, e in enumerate(step):
                qt, W, x, y, N, K = e["qtype"], e["W"], e["x"], e["y"], e["N"], e["K"]
                f16 = bool(e.get("f16", False))
                where = f"steps[{s}][{i}]"
                _weights(qt, W, N, K, where + ".W")
                if e.get("W2") is not None:
                    _weights(qt, e["W2"], N, K, where + ".W2")
                if _activations(x, K) != 1:
                    raise ValueError(f"{where}.x must be one column")
                _need(y, where + ".y", torch.float16 if f16 else torch.float32, numel=N)
                res = e.get("residual")
                if res is not None:
                    _need(res, where + ".residual", torch.float32, numel=N)
                _same_cuda_device(W=W, W2=e.get("W2"), x=x, y=y, residual=res)
                entries.append(qk_chain_entry(qt, Y_F16 if f16 else 0, W.data_ptr(),
                                              e["W2"].data_ptr() if e.get("W2") is not None else None,
                                              x.data_ptr(), y.data_ptr(), res.data_ptr() if res is not None else None,
                                              N, K))
                keep.append(e)
        nbytes = qk_chain_plan_bytes(len(sizes), len(entries))
        if nbytes < 0:
            raise ValueError("bad chain size")
        self.plan = np.zeros(nbytes, dtype=np.uint8)
        rc = qk_chain_plan(entries, sizes, self.plan)
        if rc != QK_OK:
            raise QKError(rc, "qk_chain_plan")
        dev = entries and steps[0][0]["W"].device
        self.plan_dev = torch.from_numpy(self.plan).to(dev)
        self.ws_bytes = qk_chain_workspace_bytes(len(sizes))
        self.workspace = torch.zeros(self.ws_bytes // 4, dtype=torch.int32, device=dev)
        self.nsteps = len(sizes)
        self._keep = keep

    def run(self, stream=None, timeout_us: int = 0):
        rc = qk_gemv_chain(self.plan, self.plan_dev.data_ptr(), self.workspace.data_ptr(), self.ws_bytes,
                           timeout_us, _stream_handle(stream))
        if rc != QK_OK:
            raise QKError(rc, "qk_gemv_chain")

    def status(self) -> int:
        """The workspace's flag word (synchronises): 0, or CHAIN_TIMEOUT."""
        return int(self.workspace[0].item())


# ------------------------------------------------- the attention side (torch)
# Heads are tensors [rows, heads, D] of any strides >= 0, float16 or float32:
# y of a GEMV is y.view(heads, D, ncols).permute(2, 0, 1).  Work runs, and
# what a helper allocates is allocated, on the tensors' device and on
# ``stream`` (None: that device's current stream).  These calls are a few
# microseconds on the device, so what is right is found right in a few steps
# here, and put into words only where it is not.

_torch = _f16 = None  # set by the first KVCache or Rope, which every call here takes: torch, {float16: 1, float32: 0}


def _start():
    global _torch, _f16
    if _torch is None:
        import torch
        load_library()
        _f16 = {torch.float16: 1, torch.float32: 0}
        _torch = torch
    return _torch


def _heads_arg(t, name, rows=None, heads=None, D=None):
    """The qk_heads of a tensor [rows, heads, D], checked against the sizes given (None: any)."""
    try:
        f16 = _f16[t.dtype]
        r, h, d = t.shape
        if (rows is None or r == rows) and (heads is None or h == heads) and (D is None or d == D):
            return qk_heads(t.data_ptr(), *t.stride(), f16)
    except (AttributeError, KeyError, ValueError):
        pass
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in _f16:
        raise TypeError(f"{name} must be torch.float16 or torch.float32, got {t.dtype}")
    want = ["rows" if rows is None else rows, "heads" if heads is None else heads, "D" if D is None else D]
    raise ValueError(f"{name} must have shape [{', '.join(map(str, want))}], got {tuple(t.shape)}")


def _int32_arg(t, name, shape):
    """The address of a contiguous int32 tensor of this shape (None entries: any size)."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not _torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {list(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_INT_MAX = 0x7fffffff  # ctypes takes an int's low 32 bits for a C int without a word


def _seqs_arg(rows, pages, kv_len, q_start):
    i32 = _torch.int32
    try:
        nseq, = kv_len.shape
        n, mp = pages.shape
        if rows > _INT_MAX or mp > _INT_MAX:
            raise QKError(QK_EINVAL_SHAPE, "qk_kv_seqs")
        if kv_len.dtype is i32 and pages.dtype is i32 and n == nseq and kv_len.is_contiguous() and \
                pages.is_contiguous():
            if q_start is None:
                return qk_kv_seqs(rows, nseq, mp, None, kv_len.data_ptr(), pages.data_ptr())
            if q_start.dtype is i32 and q_start.shape == (nseq + 1,) and q_start.is_contiguous():
                return qk_kv_seqs(rows, nseq, mp, q_start.data_ptr(), kv_len.data_ptr(), pages.data_ptr())
    except (AttributeError, ValueError):
        pass
    _int32_arg(kv_len, "kv_len", (None,))
    nseq = kv_len.shape[0]
    _int32_arg(pages, "pages", (nseq, None))
    _int32_arg(q_start, "q_start", (nseq + 1,))
    raise ValueError("bad sequences")


def _one_device(*tensors, names):
    """The index of the CUDA device that all of the tensors (None: absent) are on."""
    dev = tensors[0].get_device()
    if dev >= 0:
        for t in tensors:
            if t is not None and t.get_device() != dev:
                break
        else:
            return dev
    _same_cuda_device(**dict(zip(names.split(), tensors)))
    raise ValueError("all tensors must be on one device")


def _elsewhere(dev, stream):
    """None where device ``dev`` and ``stream`` are the current ones, else a context in which they are."""
    torch = _torch
    if stream is None:
        return None if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)
    import contextlib
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    if stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{dev}")
    both = contextlib.ExitStack()
    both.enter_context(torch.cuda.device(dev))
    both.enter_context(torch.cuda.stream(stream))
    return both


def _current(dev):
    """The handle of a device's current stream."""
    return _torch._C._cuda_getCurrentRawStream(dev)


class Rope:
    """Norm and rotation of query and key heads (qk_rope): inv_freq float32
    [rot_dim / 2] (None: no rotation), q_norm / k_norm float32 [D] (None: no
    norm)."""

    def __init__(self, inv_freq=None, interleaved: bool = False, q_norm=None, k_norm=None, eps: float = 1e-6):
        torch = _start()
        self.tensors = (inv_freq, q_norm, k_norm)
        for name, t in zip(("inv_freq", "q_norm", "k_norm"), self.tensors):
            if t is not None:
                _need(t, name, torch.float32)
                if t.dim() != 1:
                    raise ValueError(f"{name} must have one dimension, has {t.dim()}")
        self.D = {t.numel() for t in (q_norm, k_norm) if t is not None}
        p = [None if t is None else t.data_ptr() for t in (q_norm, k_norm, inv_freq)]
        self._c = qk_rope(*p, None, eps, 0 if inv_freq is None else 2 * inv_freq.numel(), int(interleaved))

    def arg(self, D, positions, rows):
        """The qk_rope of one call."""
        if self.D and self.D != {D}:
            raise ValueError(f"q_norm and k_norm must have {D} elements, have {sorted(self.D)}")
        if positions is None:
            return self._c
        c = qk_rope.from_buffer_copy(self._c)
        c.positions = _int32_arg(positions, "positions", (rows,))
        return c


class KVCache:
    """One layer's paged 4-bit cache (qk_kv_cache): num_pages pages of
    page_size positions.  pool: uint8 device tensor of num_pages *
    qk_kv_page_bytes(...) bytes (None: allocated here)."""

    def __init__(self, num_pages: int, n_kv_heads: int, head_dim: int, page_size: int = 64, device="cuda", pool=None):
        torch = _start()
        small = all(abs(n) <= _INT_MAX for n in (head_dim, n_kv_heads, page_size))
        pb = qk_kv_page_bytes(head_dim, n_kv_heads, page_size) if small else -1
        if pb < 0 or not 1 <= num_pages <= _INT_MAX:
            raise QKError(QK_EINVAL_SHAPE, "KVCache")
        if pool is None:
            pool = torch.empty((num_pages, pb), dtype=torch.uint8, device=device)
        _need(pool, "pool", torch.uint8, numel=num_pages * pb)
        self.pool, self.page_bytes = pool, pb
        self.num_pages, self.n_kv_heads, self.head_dim, self.page_size = num_pages, n_kv_heads, head_dim, page_size
        self._c = qk_kv_cache(pool.data_ptr(), num_pages, n_kv_heads, head_dim, page_size)


def norm_rope(rope: Rope, positions, q, k=None, q_out=None, k_out=None, stream=None):
    """Norm and rotation of q [rows, heads, D] and k [rows, kv heads, D]
    (either may be None) at ``positions`` (int32 [rows]); returns (q_out,
    k_out), float16 contiguous unless given (they may be q and k)."""
    torch = _torch
    qa = None if q is None else _heads_arg(q, "q")
    rows, hq, D = (None, 0, None) if q is None else q.shape
    ka = None if k is None and q is not None else _heads_arg(k, "k", rows, None, D)
    hk = 0
    if ka is not None:
        rows, hk, D = k.shape
    r = rope.arg(D, positions, rows)
    dev = _one_device(q if q is not None else k, k, positions, q_out, k_out, *rope.tensors,
                      names="q k positions q_out k_out inv_freq q_norm k_norm")
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return norm_rope(rope, positions, q, k, q_out, k_out)
    if q is None and q_out is not None or k is None and k_out is not None:
        raise ValueError("an output without its input")
    if q is not None and q_out is None:
        q_out = torch.empty((rows, hq, D), dtype=torch.float16, device=q.device)
    if k is not None and k_out is None:
        k_out = torch.empty((rows, hk, D), dtype=torch.float16, device=k.device)
    rc = _lib.qk_norm_rope(r, rows, D, hq, qa, None if q is None else _heads_arg(q_out, "q_out", rows, hq, D), hk, ka,
                      None if k is None else _heads_arg(k_out, "k_out", rows, hk, D), _current(dev))
    if rc != QK_OK:
        raise QKError(rc, "qk_norm_rope")
    return q_out, k_out


def kv_append(cache: KVCache, k, v, pages, kv_len, q_start=None, q=None, rope: Rope | None = None, positions=None,
              q_out=None, stream=None):
    """Keys and values [rows, kv heads, D] of new rows into the cache (see
    qk_kv_seqs: pages int32 [nseq, max_pages], kv_len int32 [nseq], q_start
    int32 [nseq + 1] or None), keys -- and the queries q [rows, heads, D] --
    normed and rotated by ``rope``; returns q_out (float16 unless given; None
    without q).  Rows of no sequence are left as they were: undefined in a
    q_out that is allocated here."""
    torch = _torch
    D, hk = cache.head_dim, cache.n_kv_heads
    ka = _heads_arg(k, "k", None, hk, D)
    rows = k.shape[0]
    va = _heads_arg(v, "v", rows, hk, D)
    qa = None if q is None else _heads_arg(q, "q", rows, None, D)
    seqs = _seqs_arg(rows, pages, kv_len, q_start)
    if rope is not None:
        r = rope.arg(D, positions, rows)
        dev = _one_device(k, v, pages, kv_len, q_start, q, q_out, cache.pool, positions, *rope.tensors,
                          names="k v pages kv_len q_start q q_out pool positions inv_freq q_norm k_norm")
    else:
        if positions is not None:
            raise ValueError("positions without a rope")
        r = None
        dev = _one_device(k, v, pages, kv_len, q_start, q, q_out, cache.pool,
                          names="k v pages kv_len q_start q q_out pool")
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return kv_append(cache, k, v, pages, kv_len, q_start, q, rope, positions, q_out)
    hq, oa = 0, None
    if q is not None:
        hq = q.shape[1]
        if q_out is None:
            q_out = torch.empty((rows, hq, D), dtype=torch.float16, device=q.device)
        oa = _heads_arg(q_out, "q_out", rows, hq, D)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rc = _lib.qk_kv_append(cache._c, seqs, r, ka, va, hq, qa, oa, _current(dev))
    if rc != QK_OK:
        raise QKError(rc, "qk_kv_append")
    return q_out


def kv_read(cache: KVCache, rows: int, pages, kv_len, q_start=None, k_out=None, v_out=None, stream=None):
    """What the cache holds at the rows' positions: (k, v), float32
    [rows, kv heads, D] unless given.  Rows of no sequence are left as they
    were."""
    torch = _torch
    seqs = _seqs_arg(rows, pages, kv_len, q_start)
    shape = (rows, cache.n_kv_heads, cache.head_dim)
    dev = _one_device(pages, kv_len, q_start, cache.pool, k_out, v_out, names="pages kv_len q_start pool k_out v_out")
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return kv_read(cache, rows, pages, kv_len, q_start, k_out, v_out)
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.float32, device=pages.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=torch.float32, device=pages.device)
    rc = _lib.qk_kv_read(cache._c, seqs, _heads_arg(k_out, "k_out", *shape), _heads_arg(v_out, "v_out", *shape),
                    _current(dev))
    if rc != QK_OK:
        raise QKError(rc, "qk_kv_read")
    return k_out, v_out


def kv_attn(cache: KVCache, q, pages, kv_len, q_start=None, scale: float | None = None, window: int = 0, out=None,
            workspace=None, stream=None):
    """Attention of q (float16 [rows, heads, D]) over the rows' sequences;
    scale None: D ** -0.5; window 0: none.  Returns out, float16 contiguous
    unless given.  workspace: uint8 device tensor of at least
    qk_kv_attn_workspace_bytes bytes (None: allocated for the call).  Rows of
    no sequence are left as they were: undefined in an out that is allocated
    here."""
    torch = _torch
    D = cache.head_dim
    qa = _heads_arg(q, "q", None, None, D)
    if not qa.f16:
        raise TypeError(f"q must be torch.float16, got {q.dtype}")
    rows, heads, _ = q.shape
    seqs = _seqs_arg(rows, pages, kv_len, q_start)
    dev = _one_device(q, pages, kv_len, q_start, out, cache.pool, workspace,
                      names="q pages kv_len q_start out pool workspace")
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return kv_attn(cache, q, pages, kv_len, q_start, scale, window, out, workspace)
    if out is None:
        out = torch.empty((rows, heads, D), dtype=torch.float16, device=q.device)
    oa = _heads_arg(out, "out", rows, heads, D)
    c = cache._c
    if workspace is None:
        need = _lib.qk_kv_attn_workspace_bytes(c, seqs, heads)
        ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need > 0 else None
    else:
        _need(workspace, "workspace", torch.uint8)
        ws, need = workspace, workspace.numel()
    window = max(-1, min(window, _INT_MAX))  # (no context is longer)
    rc = _lib.qk_kv_attn(c, seqs, heads, qa, oa, D ** -0.5 if scale is None else scale, window,
                    None if ws is None else ws.data_ptr(), max(need, 0), _current(dev))
    if rc != QK_OK:
        raise QKError(rc, "qk_kv_attn")
    return out
