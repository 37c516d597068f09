"""ctypes binding of librmt.so (include/rmt.h): the same entry points, argument marshalling only.

Every step of the ARMT prefill runs in the library's CUDA kernels. Arrays may be torch
tensors (device or host) or numpy arrays (host); pointers are passed through unchanged.
If librmt.so is missing this module raises at import: there is no fallback path. The
environment variable RMT_LIBRARY selects another build of the same ABI (librmt_debug.so,
the in-kernel bounds-checking build).
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("RMT_LIBRARY") or os.path.join(_HERE, "librmt.so")
DEBUG_LIB_PATH = os.path.join(_HERE, "librmt_debug.so")

RMT_OK, RMT_EINVAL, RMT_ENOMEM, RMT_ECUDA, RMT_ETIMEOUT, RMT_ESTATE, RMT_ERANGE, RMT_EDEBUG = range(8)
RMT_DIAGONAL, RMT_SEQUENTIAL = 0, 1
RMT_F32, RMT_BF16, RMT_BF16_SPLIT = 0, 1, 2
SCHEDULES = {"diagonal": RMT_DIAGONAL, "sequential": RMT_SEQUENTIAL}
# "bf16-split": bf16 storage, split (high + low f16 term) tensor-core operands (include/rmt.h)
DTYPES = {"f32": RMT_F32, "bf16": RMT_BF16, "bf16-split": RMT_BF16_SPLIT}
# how a cell writes its memory rows (include/rmt.h rmt_mem_update)
MEM_UPDATES = {"batched": 0, "sequential": 1}
STORAGE_BF16 = ("bf16", "bf16-split")
STATUS_NAMES = {0: "RMT_OK", 1: "RMT_EINVAL", 2: "RMT_ENOMEM", 3: "RMT_ECUDA", 4: "RMT_ETIMEOUT", 5: "RMT_ESTATE",
                6: "RMT_ERANGE", 7: "RMT_EDEBUG"}

EXPORTED = ("rmt_create", "rmt_reserve", "rmt_forward", "rmt_forward_resume", "rmt_forward_batch",
            "rmt_full_attention_forward", "rmt_schedule_table",
            "rmt_schedule_table_batch", "rmt_get_schedule", "rmt_get_trace", "rmt_sync", "rmt_wait_selftest",
            "rmt_bounds_selftest",
            "rmt_destroy", "rmt_last_error", "rmt_grouped_gemm_bf16", "rmt_attention", "rmt_memory_read",
            "rmt_memory_update", "rmt_memory_update_sequential", "rmt_memory_write", "rmt_memory_write_noalloc", "rmt_rmsnorm", "rmt_probe",
            "rmt_probe_read", "rmt_attention_window", "rmt_cache_page_bytes", "rmt_cache_write", "rmt_cache_read",
            "rmt_attention_cache_workspace", "rmt_attention_cache")

KERNELS = ("assemble", "memq", "memread", "memo", "rmsnorm1", "qkv", "attention", "o", "rmsnorm2", "gateup", "down",
           "memkv", "memupdate", "emit")


class RmtError(RuntimeError):
    def __init__(self, status: int, fn: str, msg: str):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class rmt_cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_layers", "d_model", "n_heads", "n_kv_heads", "head_dim", "d_ff",
                                               "seg_len", "n_mem", "d_k", "d_v")] + \
               [("rope_theta", ctypes.c_float), ("rms_eps", ctypes.c_float), ("mem_eps", ctypes.c_float),
                ("dtype", ctypes.c_int), ("mem_update", ctypes.c_int)]


RMT_CACHE_PAGE = 64  # tokens per page of the 4-bit key/value cache


class rmt_cache_struct(ctypes.Structure):
    """struct rmt_cache of include/rmt.h."""
    _fields_ = [("pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("lens", ctypes.c_void_p)] + \
               [(n, ctypes.c_int32) for n in ("n_pages", "n_seqs", "max_pages", "n_kv_heads", "head_dim")]


_PP = ctypes.POINTER(ctypes.c_void_p)


class rmt_weights(ctypes.Structure):
    _fields_ = [(n, _PP) for n in ("wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down", "w_mq", "w_mk", "w_mv", "w_mo",
                                   "g_attn", "g_mlp")] + [("mem_tokens", ctypes.c_void_p)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m recurrent_memory_transformer_anti_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    p32 = ctypes.POINTER(ctypes.c_int32)
    sigs = {
        "rmt_create": [ctypes.POINTER(rmt_weights), ctypes.POINTER(rmt_cfg), ctypes.POINTER(vp)],
        "rmt_forward": [vp, vp, i32, ctypes.c_int, vp, vp, vp, vp],
        "rmt_forward_resume": [vp, vp, i32, ctypes.c_int, vp, vp, vp, vp, vp, vp],
        "rmt_forward_batch": [vp, vp, i32, p32, ctypes.c_int, vp, vp, vp, vp, vp, vp],
        "rmt_reserve": [vp, i32],
        "rmt_full_attention_forward": [vp, vp, i32, vp, vp],
        "rmt_schedule_table": [i32, i32, ctypes.c_int, p32, sz],
        "rmt_schedule_table_batch": [i32, i32, p32, ctypes.c_int, p32, sz],
        "rmt_get_schedule": [vp, i32, ctypes.c_int, p32, sz],
        "rmt_get_trace": [vp, p32, sz],
        "rmt_sync": [vp, vp],
        "rmt_wait_selftest": [ctypes.c_uint32, vp],
        "rmt_bounds_selftest": [vp],
        "rmt_destroy": [vp],
        "rmt_grouped_gemm_bf16": [vp, vp, vp, i32, i32, i32, i32, ctypes.c_int, vp],
        "rmt_attention": [vp, vp, i32, i32, i32, i32, i32, ctypes.c_int, vp],
        "rmt_memory_read": [vp, vp, vp, vp, i32, i32, i32, i32, f32, ctypes.c_int, vp],
        "rmt_memory_update": [vp, vp, vp, vp, i32, i32, i32, i32, f32, vp],
        "rmt_memory_update_sequential": [vp, vp, vp, vp, i32, i32, i32, i32, f32, vp],
        "rmt_memory_write": [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, ctypes.c_int, vp],
        "rmt_memory_write_noalloc": [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, ctypes.c_int, vp],
        "rmt_rmsnorm": [vp, vp, vp, i32, i32, f32, ctypes.c_int, vp],
        "rmt_probe": [vp, ctypes.c_uint32],
        "rmt_probe_read": [vp, ctypes.c_int, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64),
                           ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double),
                           ctypes.POINTER(ctypes.c_int64)],
    }
    cache = ctypes.POINTER(rmt_cache_struct)
    sigs.update({
        "rmt_attention_window": [vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, ctypes.c_int, vp],
        "rmt_cache_page_bytes": [i32, i32],
        "rmt_cache_write": [cache, vp, vp, ctypes.c_int64, i32, vp, ctypes.c_int, vp],
        "rmt_cache_read": [cache, vp, vp, ctypes.c_int64, i32, vp, ctypes.c_int, vp],
        "rmt_attention_cache_workspace": [cache, i32, i32, i32, i32],
        "rmt_attention_cache": [cache, vp, ctypes.c_int64, vp, i32, i32, i32, i32, vp, sz, ctypes.c_int, vp],
    })
    for name, args in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = sz if name in ("rmt_cache_page_bytes", "rmt_attention_cache_workspace") else ctypes.c_int
    lib.rmt_last_error.argtypes = []
    lib.rmt_last_error.restype = ctypes.c_char_p
    return lib


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


def rmt_last_error() -> str:
    return _lib.rmt_last_error().decode()


def _check(status: int, fn: str) -> None:
    if status != RMT_OK:
        raise RmtError(status, fn, rmt_last_error())


def _ptr(x):
    """Raw address of a torch tensor / numpy array (None -> NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if isinstance(x, np.ndarray):
        if not x.flags["C_CONTIGUOUS"]:
            raise ValueError("numpy arrays must be C-contiguous")
        return x.ctypes.data
    if hasattr(x, "data_ptr"):
        if not x.is_contiguous():
            raise ValueError("tensors must be contiguous")
        return x.data_ptr()
    raise TypeError(f"cannot take the address of {type(x)}")


def _ptr32(x, count=None):
    """Raw address of an int32 array (None -> NULL), of at least `count` entries if given."""
    if x is None or isinstance(x, int):
        return x
    if "int32" not in str(x.dtype):
        raise TypeError(f"an int32 array is needed, not {x.dtype}")
    if count is not None and x.shape[0] < count:
        raise ValueError(f"{count} entries are needed, not {tuple(x.shape)}")
    return _ptr(x)


def _same_device(device: int, *arrays) -> None:
    """Refuse tensors that are not on `device` (an index; -1 is host memory): a kernel would fault on their
    addresses. Addresses and None are taken as they are."""
    for x in arrays:
        if x is not None and x.__class__ is not int:
            try:
                if x.get_device() == device:
                    continue
            except AttributeError:  # a numpy array
                pass
            raise ValueError("all tensors of a call must be on the device of its pages (or qkv)")


def _whole(x, count: int, dtype: str):
    """Address of a contiguous tensor of at least `count` values (an address is taken as it is)."""
    if x is None or isinstance(x, int):
        return x
    if _row_types.get(x.dtype) != dtype and _ROW_TYPES.get(str(x.dtype)) != dtype:
        raise TypeError(f"a tensor of type {x.dtype} given as {dtype!r}")
    if x.numel() < count:
        raise ValueError(f"{count} values are needed, not {tuple(x.shape)}")
    return _ptr(x)


def _rows(x, n: int, M: int, width: int, dtype: str):
    """Address and row stride (elements) of n * M rows of `width` values: a tensor [n, M, ...] whose rows
    are contiguous and equally spaced, possibly a slice of wider rows."""
    if _row_types.get(x.dtype) != dtype and _ROW_TYPES.get(str(x.dtype)) != dtype:
        raise TypeError(f"rows of type {x.dtype} given as {dtype!r}")
    _row_types[x.dtype] = dtype  # a lookup by name the first time only
    shape, st = x.shape, x.stride()
    if len(shape) < 3 or shape[0] != n or shape[1] != M:
        raise ValueError(f"rows must be [{n}, {M}, {width}], not {tuple(shape)}")
    ld = st[1] if M > 1 else st[0] if n > 1 else width
    ok = ld >= width and (n == 1 or st[0] == M * ld)
    if len(shape) == 3 and shape[2] == width:
        ok = ok and (st[2] == 1 or width == 1)
    else:
        if x.numel() != n * M * width:
            raise ValueError(f"rows must be [{n}, {M}, {width}], not {tuple(shape)}")
        step = 1
        for d in range(len(shape) - 1, 1, -1):
            ok = ok and (shape[d] == 1 or st[d] == step)
            step *= shape[d]
    if not ok:
        raise ValueError("rows must be contiguous and equally spaced")
    return x.data_ptr(), ld


_ROW_TYPES = {"torch.bfloat16": "bf16", "torch.float32": "f32"}
_row_types = {}  # dtype -> its name above, as far as seen


_current_stream = None  # device index -> its raw current stream, once CUDA was found available


def _stream(stream, device=None):
    """Raw stream; None: the current one of `device` (None: of the current device)."""
    if stream is None:
        global _current_stream
        if _current_stream is None:
            import torch
            if not torch.cuda.is_available():
                return None
            _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
                lambda d: torch.cuda.current_stream(d).cuda_stream)
        if device is None or device < 0:
            import torch
            device = torch.cuda.current_device()
        return _current_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def make_cfg(cfg) -> rmt_cfg:
    """rmt_cfg from an object with the ArmtConfig field names."""
    c = rmt_cfg()
    for n, _ in rmt_cfg._fields_[:10]:
        setattr(c, n, int(getattr(cfg, n)))
    c.rope_theta, c.rms_eps, c.mem_eps = float(cfg.rope_theta), float(cfg.rms_eps), float(cfg.mem_eps)
    c.dtype = DTYPES[cfg.dtype] if isinstance(cfg.dtype, str) else int(cfg.dtype)
    mu = getattr(cfg, "mem_update", "batched")
    c.mem_update = MEM_UPDATES[mu] if isinstance(mu, str) else int(mu)
    return c


class Handle:
    """An rmt_handle* together with the Python objects its creation referenced."""

    def __init__(self, ptr: int, cfg):
        self.ptr = ptr
        self.cfg = cfg

    def __del__(self):
        if getattr(self, "ptr", None) and _lib is not None:  # the module may be torn down at exit
            _lib.rmt_destroy(self.ptr)
            self.ptr = None


def rmt_create(weights: dict, cfg) -> Handle:
    """weights: {key: [per-layer arrays]} + "mem_tokens", stored in cfg.dtype (see include/rmt.h)."""
    keep = []

    def arr(key):
        ptrs = (ctypes.c_void_p * cfg.n_layers)(*[_ptr(a) for a in weights[key]])
        keep.append(ptrs)
        return ctypes.cast(ptrs, _PP)

    w = rmt_weights()
    for n, _ in rmt_weights._fields_[:-1]:
        setattr(w, n, arr(n))
    w.mem_tokens = _ptr(weights["mem_tokens"])
    c = make_cfg(cfg)
    out = ctypes.c_void_p()
    _check(_lib.rmt_create(ctypes.byref(w), ctypes.byref(c), ctypes.byref(out)), "rmt_create")
    return Handle(out.value, cfg)


def rmt_forward(h: Handle, emb, n_segments: int, schedule, out_hidden, out_A=None, out_z=None, stream=None) -> None:
    sch = SCHEDULES[schedule] if isinstance(schedule, str) else int(schedule)
    _check(_lib.rmt_forward(h.ptr, _ptr(emb), int(n_segments), sch, _ptr(out_hidden), _ptr(out_A), _ptr(out_z),
                            _stream(stream)), "rmt_forward")


def rmt_forward_resume(h: Handle, emb, n_segments: int, schedule, in_A, in_z, out_hidden, out_A=None, out_z=None,
                       stream=None) -> None:
    sch = SCHEDULES[schedule] if isinstance(schedule, str) else int(schedule)
    _check(_lib.rmt_forward_resume(h.ptr, _ptr(emb), int(n_segments), sch, _ptr(in_A), _ptr(in_z), _ptr(out_hidden),
                                   _ptr(out_A), _ptr(out_z), _stream(stream)), "rmt_forward_resume")


def rmt_forward_batch(h: Handle, emb, n_tokens, schedule, out_hidden, in_A=None, in_z=None, out_A=None, out_z=None,
                      stream=None) -> None:
    sch = SCHEDULES[schedule] if isinstance(schedule, str) else int(schedule)
    nt = np.ascontiguousarray(np.asarray(n_tokens, dtype=np.int32).reshape(-1))
    _check(_lib.rmt_forward_batch(h.ptr, _ptr(emb), int(nt.size), nt.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                  sch, _ptr(in_A), _ptr(in_z), _ptr(out_hidden), _ptr(out_A), _ptr(out_z),
                                  _stream(stream)), "rmt_forward_batch")


def rmt_full_attention_forward(h: Handle, emb, n_tokens: int, out_hidden, stream=None) -> None:
    _check(_lib.rmt_full_attention_forward(h.ptr, _ptr(emb), int(n_tokens), _ptr(out_hidden), _stream(stream)),
           "rmt_full_attention_forward")


def rmt_reserve(h: Handle, max_batch: int) -> None:
    _check(_lib.rmt_reserve(h.ptr, int(max_batch)), "rmt_reserve")


def rmt_schedule_table_batch(n_layers: int, n_segments, schedule) -> np.ndarray:
    sch = SCHEDULES[schedule] if isinstance(schedule, str) else int(schedule)
    ns = np.ascontiguousarray(np.asarray(n_segments, dtype=np.int32).reshape(-1))
    out = np.zeros(4 * n_layers * int(ns.sum()), np.int32)
    _check(_lib.rmt_schedule_table_batch(n_layers, int(ns.size), ns.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), sch,
                                         out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), out.size),
           "rmt_schedule_table_batch")
    return out.reshape(-1, 4)


def rmt_schedule_table(n_layers: int, n_segments: int, schedule) -> np.ndarray:
    sch = SCHEDULES[schedule] if isinstance(schedule, str) else int(schedule)
    out = np.zeros(3 * n_layers * n_segments, np.int32)
    _check(_lib.rmt_schedule_table(n_layers, n_segments, sch, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                   out.size), "rmt_schedule_table")
    return out.reshape(-1, 3)


def rmt_get_schedule(h: Handle, n_segments: int, schedule) -> np.ndarray:
    sch = SCHEDULES[schedule] if isinstance(schedule, str) else int(schedule)
    out = np.zeros(3 * h.cfg.n_layers * n_segments, np.int32)
    _check(_lib.rmt_get_schedule(h.ptr, n_segments, sch, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                 out.size), "rmt_get_schedule")
    return out.reshape(-1, 3)


def rmt_get_trace(h: Handle, n_cells: int) -> np.ndarray:
    out = np.zeros(3 * n_cells, np.int32)
    _check(_lib.rmt_get_trace(h.ptr, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), out.size), "rmt_get_trace")
    return out.reshape(-1, 3)


def rmt_sync(h: Handle | None, stream=None) -> None:
    """Wait for `stream` and raise what the device met (without a handle: the kernel-level entry points on the
    stream's device; a default stream's handle is 0 on every device, so that device is made the current one)."""
    device = getattr(stream, "device", None)
    if h is None and device is not None:
        import torch
        with torch.cuda.device(device):
            _check(_lib.rmt_sync(None, stream.cuda_stream), "rmt_sync")
        return
    _check(_lib.rmt_sync(h.ptr if h is not None else None, _stream(stream)), "rmt_sync")


def rmt_wait_selftest(limit_us: int, stream=None) -> None:
    _check(_lib.rmt_wait_selftest(int(limit_us), _stream(stream)), "rmt_wait_selftest")


def rmt_bounds_selftest(stream=None) -> None:
    _check(_lib.rmt_bounds_selftest(_stream(stream)), "rmt_bounds_selftest")


def rmt_destroy(h: Handle) -> None:
    if h.ptr:
        _check(_lib.rmt_destroy(h.ptr), "rmt_destroy")
        h.ptr = None


def rmt_probe(h: Handle, kernels=()) -> None:
    """Time every launch of the named kernel kinds (see KERNELS) in later forwards."""
    mask = 0
    for k in kernels:
        mask |= 1 << KERNELS.index(k)
    _check(_lib.rmt_probe(h.ptr, mask), "rmt_probe")


def rmt_probe_read(h: Handle, kernel: str) -> dict:
    ms, fl, by = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
    nl, al = ctypes.c_int64(), ctypes.c_int64()
    _check(_lib.rmt_probe_read(h.ptr, KERNELS.index(kernel), ctypes.byref(ms), ctypes.byref(nl), ctypes.byref(fl),
                               ctypes.byref(by), ctypes.byref(al)), "rmt_probe_read")
    return {"ms": ms.value, "launches": nl.value, "flops": fl.value, "bytes": by.value, "all_launches": al.value}


def rmt_grouped_gemm_bf16(A, B, C, G, M, N, K, out_dtype="f32", stream=None) -> None:
    _check(_lib.rmt_grouped_gemm_bf16(_ptr(A), _ptr(B), _ptr(C), G, M, N, K, DTYPES[out_dtype], _stream(stream)),
           "rmt_grouped_gemm_bf16")


def rmt_attention(qkv, out, G, M, H, Hkv, dh, dtype="bf16", stream=None) -> None:
    _check(_lib.rmt_attention(_ptr(qkv), _ptr(out), G, M, H, Hkv, dh, DTYPES[dtype], _stream(stream)), "rmt_attention")


def rmt_memory_read(q, A, z, o, G, M, dk, dv, eps, dtype="f32", stream=None) -> None:
    _check(_lib.rmt_memory_read(_ptr(q), _ptr(A), _ptr(z), _ptr(o), G, M, dk, dv, eps, DTYPES[dtype],
                                _stream(stream)), "rmt_memory_read")


def rmt_memory_update(k, v, A, z, G, n, dk, dv, eps, stream=None) -> None:
    _check(_lib.rmt_memory_update(_ptr(k), _ptr(v), _ptr(A), _ptr(z), G, n, dk, dv, eps, _stream(stream)),
           "rmt_memory_update")


def rmt_memory_update_sequential(k, v, A, z, G, n, dk, dv, eps, stream=None) -> None:
    _check(_lib.rmt_memory_update_sequential(_ptr(k), _ptr(v), _ptr(A), _ptr(z), G, n, dk, dv, eps,
                                             _stream(stream)), "rmt_memory_update_sequential")


def rmt_memory_write(y, w_mkv, A, z, G, n, d, dk, dv, eps, dtype="f32", stream=None) -> None:
    _check(_lib.rmt_memory_write(_ptr(y), _ptr(w_mkv), _ptr(A), _ptr(z), G, n, d, dk, dv, eps, DTYPES[dtype],
                                 _stream(stream)), "rmt_memory_write")


def rmt_memory_write_noalloc(y, w_mkv, A, z, G, n, d, dk, dv, eps, dtype="f32", stream=None) -> None:
    """rmt_memory_write with its scratch in the library's fixed device array (no cudaMalloc)."""
    _check(_lib.rmt_memory_write_noalloc(_ptr(y), _ptr(w_mkv), _ptr(A), _ptr(z), G, n, d, dk, dv, eps,
                                         DTYPES[dtype], _stream(stream)), "rmt_memory_write_noalloc")


def rmt_rmsnorm(x, g, y, rows, d, eps, dtype="f32", stream=None) -> None:
    _check(_lib.rmt_rmsnorm(_ptr(x), _ptr(g), _ptr(y), rows, d, eps, DTYPES[dtype], _stream(stream)), "rmt_rmsnorm")


def rmt_attention_window(qkv, out, G, M, H, Hkv, dh, window, sinks=0, lens=None, dtype="bf16", stream=None) -> None:
    """Attention over a sliding window (0: none) and the first `sinks` tokens; lens: int32 [G] on the device or None."""
    device = None
    if not isinstance(qkv, int):
        device = qkv.get_device()
        _same_device(device, out, lens)
    _check(_lib.rmt_attention_window(_whole(qkv, G * M * (H + 2 * Hkv) * dh, dtype), _whole(out, G * M * H * dh, dtype),
                                     G, M, H, Hkv, dh, window, sinks, _ptr32(lens, G), DTYPES[dtype],
                                     _stream(stream, device)), "rmt_attention_window")


class Cache:
    """An rmt_cache (include/rmt.h) together with the tensors it points to."""

    def __init__(self, struct: rmt_cache_struct, keep: tuple):
        self.struct = struct
        self.keep = keep
        self.ref = ctypes.byref(struct)
        self.n_seqs, self.head_dim = struct.n_seqs, struct.head_dim
        self.width = struct.n_kv_heads * struct.head_dim
        self.device = keep[0].get_device()


def rmt_cache_page_bytes(n_kv_heads: int, head_dim: int) -> int:
    n = _lib.rmt_cache_page_bytes(n_kv_heads, head_dim)
    if n == 0:
        raise ValueError(f"no cache page for {n_kv_heads} heads of {head_dim}")
    return n


def rmt_cache(pages, page_table, lens, n_kv_heads: int, head_dim: int) -> Cache:
    """The 4-bit key/value cache in these device tensors: pages (uint8, whole pages), page_table (int32
    [n_seqs, max_pages]) and lens (int32 [n_seqs]). Their contents may change between calls."""
    size = pages.numel() * pages.element_size()
    page = rmt_cache_page_bytes(n_kv_heads, head_dim)
    if size % page or page_table.ndim != 2 or lens.ndim != 1 or lens.shape[0] != page_table.shape[0]:
        raise ValueError(f"pages must hold whole pages of {page} bytes, page_table [n_seqs, max_pages] and lens [n_seqs]")
    _same_device(pages.get_device(), page_table, lens)
    s = rmt_cache_struct(_ptr(pages), _ptr32(page_table), _ptr32(lens), size // page, page_table.shape[0],
                         page_table.shape[1], n_kv_heads, head_dim)
    return Cache(s, (pages, page_table, lens))


def _cache_rows(fn, name, cache, k, v, M, n_new, dtype, stream):
    _same_device(cache.device, k, v, n_new)
    pk, ld = _rows(k, cache.n_seqs, M, cache.width, dtype)
    if v.dtype is k.dtype and v.shape == k.shape and v.stride() == k.stride():
        pv = v.data_ptr()
    else:
        pv, ldv = _rows(v, cache.n_seqs, M, cache.width, dtype)
        if ld != ldv:
            raise ValueError("k and v need the same row stride")
    _check(fn(cache.ref, pk, pv, ld, M, _ptr32(n_new, cache.n_seqs), DTYPES[dtype],
              _stream(stream, cache.device)), name)


def rmt_cache_write(cache: Cache, k, v, M, n_new=None, dtype="bf16", stream=None) -> None:
    """Quantise rows k, v ([n_seqs, M, n_kv_heads * head_dim], views into wider rows allowed) into the cache."""
    _cache_rows(_lib.rmt_cache_write, "rmt_cache_write", cache, k, v, M, n_new, dtype, stream)


def rmt_cache_read(cache: Cache, k, v, M, n_new=None, dtype="bf16", stream=None) -> None:
    """The values the cache holds for the rows rmt_cache_write takes, into k, v."""
    _cache_rows(_lib.rmt_cache_read, "rmt_cache_read", cache, k, v, M, n_new, dtype, stream)


def rmt_attention_cache_workspace(cache: Cache, n_q: int, H: int, window: int = 0, sinks: int = 0) -> int:
    n = _lib.rmt_attention_cache_workspace(cache.ref, n_q, H, window, sinks)
    if n == 0:
        raise RmtError(RMT_EINVAL, "rmt_attention_cache_workspace", rmt_last_error())
    return n


def rmt_attention_cache(cache: Cache, q, out, n_q, H, window, sinks, workspace, dtype="bf16", stream=None) -> None:
    """Attention of the newest n_q tokens of each sequence (q rows [n_seqs, n_q, H * head_dim], a view into
    wider rows allowed) over the cache. workspace: a uint8 tensor of rmt_attention_cache_workspace bytes."""
    _same_device(cache.device, q, out, workspace)
    pq, ldq = _rows(q, cache.n_seqs, n_q, H * cache.head_dim, dtype)
    _check(_lib.rmt_attention_cache(cache.ref, pq, ldq, _whole(out, cache.n_seqs * n_q * H * cache.head_dim, dtype),
                                    n_q, H, window, sinks,
                                    _ptr(workspace), workspace.numel() * workspace.element_size(), DTYPES[dtype],
                                    _stream(stream, cache.device)), "rmt_attention_cache")


def storage(a, dtype: str, device=None):
    """A float32 array as a torch tensor in the model's storage dtype (marshalling helper)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    t = t.to(torch.bfloat16) if dtype in STORAGE_BF16 else t
    return t.to(device) if device is not None else t


def weights_storage(weights: dict, dtype: str, device=None) -> dict:
    return {k: ([storage(a, dtype, device) for a in v] if isinstance(v, list) else storage(v, dtype, device))
            for k, v in weights.items()}
