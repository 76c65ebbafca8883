"""Python binding of libdcp: decode attention over a sequence-sharded paged KV
cache (Decode Context Parallelism) on NVIDIA B200.

This module only marshals arguments: torch tensors become device pointers,
the current torch stream becomes the cudaStream_t, and a non-zero status
becomes :class:`DcpError`.  Every step of the path runs in the CUDA kernels of
``libdcp.so`` (built in-tree from ``csrc/`` by ``build.py``).  There is no
fallback: if the library is missing, importing the entry points raises.

Entry points (same names as ``include/dcp.h``): ``dcp_shard_counts``,
``dcp_shard_map``, ``dcp_kv_append``, ``dcp_decode_workspace_size``,
``dcp_decode_workspace_size_ex``, ``dcp_decode_partial``,
``dcp_decode_partial_multi``, ``dcp_decode_merged``,
``dcp_decode_partial_noalloc``, ``dcp_merge``, ``dcp_get_device_status``,
``dcp_norm_rope_append`` (with ``make_rope``), ``dcp_kv_gather``,
``dcp_decode_window``, and for one rank of a multi-GPU group ``dcp_kv_append_rank``, ``dcp_decode_rank``,
``dcp_lse_rescale`` (the collectives around them are in ``parallel.py``).
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdcp.so")

DCP_OK = 0
DCP_ERR_INVALID_ARG = 1
DCP_ERR_UNSUPPORTED = 2
DCP_ERR_UNALLOCATED_PAGE = 3
DCP_ERR_WORKSPACE_TOO_SMALL = 4
DCP_ERR_CUDA = 5
DCP_ERR_MISALIGNED = 6
DCP_ERR_TIMEOUT = 7

DCP_GQA = 0
DCP_MLA = 1
DCP_BF16 = 0
DCP_FP8_E4M3 = 1
DCP_FP4_E2M1 = 2

DCP_ROPE_HALF = 0
DCP_ROPE_INTERLEAVED = 1
ROPE_SCALINGS = ("none", "linear", "base", "yarn", "smooth")  # dcp_rope_scaling, in order

DCP_DECODE_PARTIAL = 0
DCP_DECODE_MERGED = 1
DCP_DECODE_RANK = 2

EXPORTED = ("dcp_status_string", "dcp_shard_counts", "dcp_shard_map", "dcp_kv_append",
            "dcp_decode_workspace_size", "dcp_decode_workspace_size_ex", "dcp_decode_partial",
            "dcp_decode_partial_multi", "dcp_decode_merged", "dcp_decode_partial_noalloc", "dcp_merge",
            "dcp_get_device_status", "dcp_kv_append_rank", "dcp_decode_rank", "dcp_lse_rescale", "dcp_kv_gather",
            "dcp_rope_init", "dcp_norm_rope_append", "dcp_decode_window", "dcp_decode_window_workspace_size")


class DcpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class CacheDesc(ctypes.Structure):
    """Mirror of ``dcp_cache_desc``."""
    _fields_ = [
        ("kind", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("n_shards", ctypes.c_int32), ("interleave", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("batch", ctypes.c_int32), ("max_local_pages", ctypes.c_int32), ("reserved0", ctypes.c_int32),
        ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
        ("kv_scales", ctypes.c_void_p), ("block_tables", ctypes.c_void_p),
    ]


class Rope(ctypes.Structure):
    """Mirror of ``dcp_rope`` (host memory; filled by :func:`dcp_rope_init`)."""
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("attn_factor", ctypes.c_float),
                ("reserved0", ctypes.c_int32), ("turns", ctypes.c_uint64 * 64)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libdcp.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libdcp.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        D = ctypes.POINTER(CacheDesc)
        L.dcp_status_string.argtypes = [ctypes.c_int]
        L.dcp_status_string.restype = ctypes.c_char_p
        L.dcp_shard_counts.argtypes = [i32, P, i32, i32, P, P]
        L.dcp_shard_map.argtypes = [D, i64, P, P, P, P, P, P]
        L.dcp_kv_append.argtypes = [D, i64, P, P, P, P, P]
        L.dcp_decode_workspace_size.argtypes = [D, i32]
        L.dcp_decode_workspace_size.restype = ctypes.c_size_t
        L.dcp_decode_partial.argtypes = [D, i32, P, P, P, P, P, ctypes.c_size_t, P]
        L.dcp_decode_workspace_size_ex.argtypes = [D, i32, i32, i32]
        L.dcp_decode_workspace_size_ex.restype = ctypes.c_size_t
        L.dcp_decode_partial_multi.argtypes = [D, i32, i32, P, P, P, P, P, ctypes.c_size_t, P]
        L.dcp_decode_merged.argtypes = [D, i32, i32, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.dcp_kv_append_rank.argtypes = [D, i32, i64, P, P, P, P, P]
        L.dcp_decode_rank.argtypes = [D, i32, i32, i32, P, P, P, P, P, ctypes.c_size_t, P]
        L.dcp_lse_rescale.argtypes = [i32, i32, i32, i32, i32, P, P, P, P, P]
        F64 = ctypes.c_double
        R = ctypes.POINTER(Rope)
        L.dcp_kv_gather.argtypes = [D, i32, i64, P, P, P, P, P]
        L.dcp_rope_init.argtypes = [R, i32, i32, F64, i32, F64, F64, F64, F64, F64]
        L.dcp_norm_rope_append.argtypes = [D, i32, R, i64, P, P, P, i64, P, i64, P, i64, P, P, ctypes.c_float, P, P]
        L.dcp_decode_window.argtypes = [D, i32, i32, i32, i32, i32, P, P, P, P, P, ctypes.c_size_t, P]
        L.dcp_decode_window_workspace_size.argtypes = [D, i32, i32, i32, i32, i32]
        L.dcp_decode_window_workspace_size.restype = ctypes.c_size_t
        L.dcp_decode_partial_noalloc.argtypes = [D, i32, P, P, P, P, P]
        L.dcp_merge.argtypes = [i32, i32, i32, i32, P, P, P, P, P]
        L.dcp_get_device_status.argtypes = [ctypes.POINTER(i32), P]
        L.dcp_selftest_bounded_wait.argtypes = [P, P]
        for name in ("dcp_shard_counts", "dcp_shard_map", "dcp_kv_append", "dcp_decode_partial",
                     "dcp_decode_partial_multi", "dcp_decode_merged", "dcp_decode_partial_noalloc", "dcp_merge",
                     "dcp_get_device_status", "dcp_kv_append_rank", "dcp_decode_rank", "dcp_lse_rescale",
                     "dcp_selftest_bounded_wait", "dcp_kv_gather", "dcp_rope_init", "dcp_norm_rope_append",
                     "dcp_decode_window"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().dcp_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        device = _device()
        if device >= 0:  # current_stream() builds a Stream object each time
            return _torch._C._cuda_getCurrentRawStream(device)
        return _torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(status: int, where: str):
    if status != DCP_OK:
        raise DcpError(status, where)


def make_cache_desc(*, kind: int, dtype: int, n_shards: int, interleave: int, page_size: int, num_pages: int,
                    hq: int, hkv: int, dk: int, dv: int, scale: float, batch: int, block_tables,
                    k_pages=None, v_pages=None, kv_scales=None) -> CacheDesc:
    """Build a ``dcp_cache_desc`` from torch tensors (block_tables int32
    [N][B][max_local_pages]); the tensors must outlive every call using it."""
    return CacheDesc(kind, dtype, n_shards, interleave, page_size, num_pages, hq, hkv, dk, dv, float(scale), batch,
                     int(block_tables.shape[2]), 0, _ptr(k_pages), _ptr(v_pages), _ptr(kv_scales),
                     _ptr(block_tables))


_torch = None  # the module, once a tensor has been checked


def _device() -> int:
    """The current device (a tensor on a GPU is at hand: torch has initialised CUDA)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch._C._cuda_getDevice() if _torch.cuda.is_initialized() else -1


def _workspace(ws, device: int) -> int:
    """Bytes of a workspace; refuse one that the kernels could not write."""
    if ws.get_device() != device or device < 0:
        raise ValueError(f"ws is on {ws.device}, not on the current CUDA device")
    if not ws.is_contiguous():
        raise ValueError(f"ws is a view with strides {ws.stride()}, not contiguous")
    return ws.numel() * ws.element_size()


def _decode_workspace(desc: CacheDesc, ws) -> int:
    """Bytes of a decode call's workspace, checked where the cache is a 4-bit one."""
    if desc.dtype == DCP_FP4_E2M1:
        return _workspace(ws, _device())
    return ws.numel() * ws.element_size()


def dcp_shard_counts(seq_lens, n_shards: int, interleave: int, counts_out, stream=None) -> None:
    _check(lib().dcp_shard_counts(seq_lens.numel(), _ptr(seq_lens), n_shards, interleave, _ptr(counts_out),
                                  _stream(stream)), "dcp_shard_counts")


def dcp_shard_map(desc: CacheDesc, pos, req, rank_out, local_out, slot_out, stream=None) -> None:
    _check(lib().dcp_shard_map(ctypes.byref(desc), pos.numel(), _ptr(pos), _ptr(req), _ptr(rank_out),
                               _ptr(local_out), _ptr(slot_out), _stream(stream)), "dcp_shard_map")


def dcp_kv_append(desc: CacheDesc, req, pos, k_new, v_new=None, stream=None) -> None:
    _check(lib().dcp_kv_append(ctypes.byref(desc), pos.numel(), _ptr(req), _ptr(pos), _ptr(k_new), _ptr(v_new),
                               _stream(stream)), "dcp_kv_append")


def dcp_decode_workspace_size(desc: CacheDesc, batch: int) -> int:
    return int(lib().dcp_decode_workspace_size(ctypes.byref(desc), batch))


def dcp_decode_partial(desc: CacheDesc, q, seq_lens, o_partial, lse, ws, stream=None) -> None:
    _check(lib().dcp_decode_partial(ctypes.byref(desc), q.shape[0], _ptr(q), _ptr(seq_lens), _ptr(o_partial),
                                    _ptr(lse), _ptr(ws), _decode_workspace(desc, ws), _stream(stream)),
           "dcp_decode_partial")


def dcp_decode_workspace_size_ex(desc: CacheDesc, batch: int, q_len: int = 1, mode: int = DCP_DECODE_PARTIAL) -> int:
    """Workspace bytes of the decode call of `mode` (DCP_DECODE_PARTIAL, _MERGED or _RANK)."""
    return int(lib().dcp_decode_workspace_size_ex(ctypes.byref(desc), batch, q_len, int(mode)))


def dcp_decode_partial_multi(desc: CacheDesc, q, seq_lens, o_partial, lse, ws, stream=None) -> None:
    """q bf16 [B][q_len][hq][dk] -> o_partial [N][B][q_len][hq][dv], lse [N][B][q_len][hq]."""
    _check(lib().dcp_decode_partial_multi(ctypes.byref(desc), q.shape[0], q.shape[1], _ptr(q), _ptr(seq_lens),
                                          _ptr(o_partial), _ptr(lse), _ptr(ws), _decode_workspace(desc, ws),
                                          _stream(stream)), "dcp_decode_partial_multi")


def dcp_decode_merged(desc: CacheDesc, q, seq_lens, out, lse_out, ws, finish_ns=None, stream=None) -> None:
    """Partial attention of every shard and the LSE merge in one launch sequence.
    q bf16 [B][hq][dk] (one query token) or [B][q_len][hq][dk]; out / lse_out have
    q's leading dimensions with dv / no trailing dimension; finish_ns int64 [B] or None."""
    q_len = 1 if q.dim() == 3 else q.shape[1]
    _check(lib().dcp_decode_merged(ctypes.byref(desc), q.shape[0], q_len, _ptr(q), _ptr(seq_lens), _ptr(out),
                                   _ptr(lse_out), _ptr(finish_ns), _ptr(ws), _decode_workspace(desc, ws),
                                   _stream(stream)), "dcp_decode_merged")


def dcp_kv_append_rank(desc: CacheDesc, rank: int, req, pos, k_new, v_new=None, stream=None) -> None:
    _check(lib().dcp_kv_append_rank(ctypes.byref(desc), rank, pos.numel(), _ptr(req), _ptr(pos), _ptr(k_new),
                                    _ptr(v_new), _stream(stream)), "dcp_kv_append_rank")


def dcp_decode_rank(desc: CacheDesc, rank: int, q, seq_lens, o, lse, ws, stream=None) -> None:
    """Rank `rank`'s partial: q bf16 [B][hq][dk] or [B][q_len][hq][dk] -> o, lse with q's leading dims."""
    q_len = 1 if q.dim() == 3 else q.shape[1]
    _check(lib().dcp_decode_rank(ctypes.byref(desc), rank, q.shape[0], q_len, _ptr(q), _ptr(seq_lens), _ptr(o),
                                 _ptr(lse), _ptr(ws), _decode_workspace(desc, ws), _stream(stream)),
           "dcp_decode_rank")


def dcp_lse_rescale(lse_all, rank: int, o, o_rs, lse_out=None, stream=None) -> None:
    """lse_all [N][B][H], o [B][H][Dv] -> o_rs [N][B][H/N][Dv] (reduce-scatter layout), lse_out [B][H]."""
    N, B, H = lse_all.shape
    _check(lib().dcp_lse_rescale(N, rank, B, H, o.shape[-1], _ptr(lse_all), _ptr(o), _ptr(o_rs), _ptr(lse_out),
                                 _stream(stream)), "dcp_lse_rescale")


def _tensor(name: str, t, device: int, dtype, shape=None) -> None:
    """Refuse a tensor whose layout the kernels would misread."""
    if t.get_device() != device or device < 0:
        raise ValueError(f"{name} is on {t.device}, not on the current CUDA device")
    if t.dtype is not dtype:
        raise ValueError(f"{name} is {t.dtype}, not {dtype}")
    if shape is not None and (t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{name} is {tuple(t.shape)} (strides {t.stride()}), not a contiguous {tuple(shape)}")


def _rank(rank) -> int:
    return -1 if rank is None else int(rank)


def _tokens(desc: CacheDesc, req, pos, device: int) -> int:
    n = pos.shape[0]
    _tensor("pos", pos, device, _torch.int32, (n,))
    if req is not None:
        _tensor("req", req, device, _torch.int32, (n,))
    elif n > desc.batch:
        raise ValueError(f"{n} tokens without req: row i belongs to request i of {desc.batch}")
    return n


def dcp_kv_gather(desc: CacheDesc, req, pos, k_out, v_out=None, rank=None, stream=None) -> None:
    """Read rows back as bf16: k_out [n][hkv][dk] (MLA [n][576]), v_out alike or None."""
    device = _device()
    n = _tokens(desc, req, pos, device)
    shape = (n, desc.hkv, desc.dk) if desc.kind == DCP_GQA else (n, desc.dk)
    _tensor("k_out", k_out, device, _torch.bfloat16, shape)
    if v_out is not None:
        _tensor("v_out", v_out, device, _torch.bfloat16, shape)
    _check(lib().dcp_kv_gather(ctypes.byref(desc), _rank(rank), n, _ptr(req), _ptr(pos), _ptr(k_out), _ptr(v_out),
                               _stream(stream)), "dcp_kv_gather")


def dcp_rope_init(rope: Rope, rot_dim: int, layout: int, theta: float, scaling: int = 0, factor: float = 1.0,
                  original: float = 0.0, low: float = 0.0, high: float = 0.0, attn_factor: float = 0.0) -> None:
    _check(lib().dcp_rope_init(ctypes.byref(rope), rot_dim, layout, theta, scaling, factor, original, low, high,
                               attn_factor), "dcp_rope_init")


def make_rope(rot_dim: int, *, layout: str = "half", theta: float = 1e4, scaling: str = "none", factor: float = 1.0,
              original: float = 0.0, low: float = 1.0, high: float = 32.0, attn_factor: float = 0.0) -> Rope:
    """A position rotation for dcp_norm_rope_append: layout "half" or "interleaved", scaling one of
    ``ROPE_SCALINGS`` (include/dcp.h says what each does with factor, original, low and high)."""
    layouts = {"half": DCP_ROPE_HALF, "interleaved": DCP_ROPE_INTERLEAVED}
    if layout not in layouts or scaling not in ROPE_SCALINGS:
        raise ValueError(f"unknown rotary layout {layout!r} or scaling {scaling!r}")
    rope = Rope()
    dcp_rope_init(rope, rot_dim, layouts[layout], theta, ROPE_SCALINGS.index(scaling), factor, original, low, high,
                  attn_factor)
    return rope


def _rows(name: str, t, device: int, shape) -> int:
    """Token stride (elements) of rows [n][..] whose inner dimensions are contiguous."""
    _tensor(name, t, device, _torch.bfloat16)
    if t.shape != shape:
        raise ValueError(f"{name} is {tuple(t.shape)}, not {tuple(shape)}")
    strides = t.stride()
    row = shape[1] * shape[2] if len(shape) == 3 else shape[1]
    if strides[-1] != 1 or (len(shape) == 3 and shape[1] > 1 and strides[1] != shape[2]):
        raise ValueError(f"{name}: a token's row is not contiguous (strides {strides})")
    return strides[0] if shape[0] > 1 else row


def dcp_norm_rope_append(desc: CacheDesc, rope, req, pos, q, k, v, q_weight, k_weight, eps: float, q_out, rank=None,
                         stream=None) -> None:
    """Per-head norms, position rotation and append in one pass.

    q bf16 [n][hq][dk], k / v bf16 [n][hkv][dk] (MLA: k [n][576], v None), rows may be strided by token (slices of
    one projection's output); q_weight / k_weight bf16 [dk] (MLA: None and [512]) or None for no norm; rope from
    make_rope or None; q_out bf16 [n][hq][dk], which may be q itself.  q and q_out, or k and v, may be None."""
    device = _device()
    n = _tokens(desc, req, pos, device)
    mla = desc.kind == DCP_MLA
    hq, hkv, dk = desc.hq, desc.hkv, desc.dk
    qs = ks = vs = 0
    if q is not None:
        qs = _rows("q", q, device, (n, hq, dk))
        if q_out is None:
            raise ValueError("q without q_out")
        _tensor("q_out", q_out, device, _torch.bfloat16, (n, hq, dk))
    kv_shape = (n, dk) if mla else (n, hkv, dk)
    if k is not None:
        ks = _rows("k", k, device, kv_shape)
    if v is not None:
        vs = _rows("v", v, device, kv_shape)
    if q_weight is not None:
        _tensor("q_weight", q_weight, device, _torch.bfloat16, (dk,))
    if k_weight is not None:
        _tensor("k_weight", k_weight, device, _torch.bfloat16, (512 if mla else dk,))
    _check(lib().dcp_norm_rope_append(ctypes.byref(desc), _rank(rank), None if rope is None else ctypes.byref(rope), n,
                                      _ptr(req), _ptr(pos), _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(q_weight),
                                      _ptr(k_weight), eps, _ptr(q_out if q is not None else None), _stream(stream)),
           "dcp_norm_rope_append")


def dcp_decode_window_workspace_size(desc: CacheDesc, batch: int, q_len: int, window: int, n_sinks: int = 0,
                                     rank=None) -> int:
    return int(lib().dcp_decode_window_workspace_size(ctypes.byref(desc), _rank(rank), batch, q_len, window, n_sinks))


def dcp_decode_window(desc: CacheDesc, q, seq_lens, window: int, n_sinks: int, out, lse, ws, rank=None,
                      stream=None) -> None:
    """Decode attention under a sliding window of `window` positions and `n_sinks` first tokens.
    q bf16 [B][hq][dk] or [B][q_len][hq][dk]; out / lse fp32 with q's leading dimensions; rank None: all shards
    merged, r: rank r's partial of a multi-GPU group."""
    device, shape, hq = _device(), q.shape, desc.hq
    B, q_len = shape[0], 1 if len(shape) == 3 else shape[1]
    lead = (B, hq) if len(shape) == 3 else (B, q_len, hq)
    f32 = _torch.float32
    _tensor("q", q, device, _torch.bfloat16, lead + (desc.dk,))
    _tensor("seq_lens", seq_lens, device, _torch.int32, (B,))
    _tensor("out", out, device, f32, lead + (desc.dv,))
    _tensor("lse", lse, device, f32, lead)
    ws_bytes = _workspace(ws, device)
    _check(lib().dcp_decode_window(ctypes.byref(desc), _rank(rank), B, q_len, window, n_sinks, _ptr(q),
                                   _ptr(seq_lens), _ptr(out), _ptr(lse), _ptr(ws), ws_bytes, _stream(stream)),
           "dcp_decode_window")


# size of the library's built-in decode scratch (DCP_STATIC_SCRATCH_BYTES in dcp.h)
DCP_STATIC_SCRATCH_BYTES = 64 << 20


def dcp_decode_partial_noalloc(desc: CacheDesc, q, seq_lens, o_partial, lse, stream=None) -> None:
    """dcp_decode_partial on the library's built-in scratch; allocates nothing.
    Calls that can overlap in time race on that scratch."""
    _check(lib().dcp_decode_partial_noalloc(ctypes.byref(desc), q.shape[0], _ptr(q), _ptr(seq_lens),
                                            _ptr(o_partial), _ptr(lse), _stream(stream)),
           "dcp_decode_partial_noalloc")


def dcp_merge(o_partial, lse, out, lse_out=None, stream=None) -> None:
    N, B, H, Dv = o_partial.shape
    _check(lib().dcp_merge(N, B, H, Dv, _ptr(o_partial), _ptr(lse), _ptr(out), _ptr(lse_out), _stream(stream)),
           "dcp_merge")


def dcp_selftest_bounded_wait(result, stream=None) -> None:
    """Launches the bounded-wait self-test: result int64 [>= 3] on the device receives
    (wait completed?, abort flag, nanoseconds waited); the status word then holds DCP_ERR_TIMEOUT."""
    _check(lib().dcp_selftest_bounded_wait(_ptr(result), _stream(stream)), "dcp_selftest_bounded_wait")


def dcp_get_device_status(stream=None) -> int:
    v = ctypes.c_int32(0)
    _check(lib().dcp_get_device_status(ctypes.byref(v), _stream(stream)), "dcp_get_device_status")
    return int(v.value)
