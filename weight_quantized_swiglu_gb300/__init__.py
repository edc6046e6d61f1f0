"""Weight-quantized SwiGLU MLP for GB300 (sm_103a): thin Python binding.

Every step of the computation runs in the CUDA kernels of ``libqmlp.so``
(built in-tree by ``weight_quantized_swiglu_gb300.build``); this module only
marshals arguments through the C ABI declared in ``include/qmlp.h``. There is
no CPU fallback: if the library is missing or fails to load, every call
raises ``RuntimeError``, and a failed call raises ``QmlpError`` (a
``RuntimeError``) carrying the library's status.

Module-level functions carry the C names (``qmlp_create``, ``qmlp_forward``,
...); ``QuantMLP`` and ``MoeAWQ`` wrap the handles for convenience. Device
buffers are passed as torch CUDA tensors (or raw integer addresses); streams
as ``torch.cuda.Stream`` (or raw handles, 0 = legacy default stream).
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libqmlp.so")

QMLP_OK = 0
STATUS = {0: "QMLP_OK", 1: "QMLP_ERR_INVALID_ARG", 2: "QMLP_ERR_ALIGNMENT", 3: "QMLP_ERR_ALIAS",
          4: "QMLP_ERR_SHAPE", 5: "QMLP_ERR_UNSUPPORTED_ARCH", 6: "QMLP_ERR_OOM", 7: "QMLP_ERR_CUDA",
          8: "QMLP_ERR_DEVICE_TIMEOUT", 9: "QMLP_ERR_DEVICE_BOUNDS"}
FMT_NVFP4, FMT_FP8_PC = 1, 2
DT_BF16, DT_FP16, DT_FP32 = 1, 2, 3
STATE_FP32, STATE_8BIT = 1, 2
META_3B, META_4B = 3, 4
PATH_AUTO, PATH_GEMV, PATH_GEMM, PATH_GEMM_PAIR, PATH_GEMM_DQ = 0, 1, 2, 3, 4


class QmlpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class qmlp_proj(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("global_scale", ctypes.c_float)]


class qmlp_desc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("K", ctypes.c_int), ("I", ctypes.c_int), ("max_M", ctypes.c_int),
                ("gate", qmlp_proj), ("up", qmlp_proj), ("down", qmlp_proj)]


class qmlp_moe_desc(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int), ("K", ctypes.c_int), ("I", ctypes.c_int), ("meta", ctypes.c_int),
                ("w13", ctypes.c_void_p), ("w13_meta", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("w2_meta", ctypes.c_void_p)]


ADAPTER_PARTS = ("gate_a", "gate_b", "up_a", "up_b", "down_a", "down_b")


class qmlp_adapter(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int), ("scale", ctypes.c_float)] + [(n, ctypes.c_void_p) for n in ADAPTER_PARTS]


class qmlp_adamw_tensor(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("param", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class qmlp_adamw_hyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("step", ctypes.c_int64)]


_lock = threading.Lock()
_lib = None

_VP = ctypes.c_void_p
_I = ctypes.c_int
_SIGS = {
    "qmlp_create": ([ctypes.POINTER(_VP), ctypes.POINTER(qmlp_desc), _VP], _I),
    "qmlp_destroy": ([_VP], None),
    "qmlp_forward": ([_VP, _VP, _I, _VP, _VP], _I),
    "qmlp_forward_path": ([_VP, _I, _VP, _I, _VP, _VP], _I),
    "qmlp_forward_host": ([_VP, _VP, _I, _VP, _VP], _I),
    "qmlp_forward_stage": ([_VP, _I, _I, _VP, _I, _VP, _VP], _I),
    "qmlp_forward_debug": ([_VP, _I, _VP, _I, _VP, _VP, _VP], _I),
    "qmlp_debug_project": ([_VP, _I, _I, _VP, _I, _VP, _VP], _I),
    "qmlp_check": ([_VP, _VP], _I),
    "qmlp_debug_split": ([_VP, _VP, _VP, _I, _VP, _VP, _VP, _VP], _I),
    "qmlp_debug_set_wait": ([_VP, ctypes.c_uint64, _I], _I),
    "qmlp_debug_bounds_enabled": ([], _I),
    "qmlp_debug_bounds": ([ctypes.POINTER(_I), ctypes.POINTER(ctypes.c_ulonglong)], _I),
    "qmlp_debug_bounds_limit": ([_VP, ctypes.c_size_t], _I),
    "qmlp_create_shard": ([ctypes.POINTER(_VP), ctypes.POINTER(qmlp_desc), _I, _I, _VP], _I),
    "qmlp_forward_partial": ([_VP, _VP, _I, _VP, _VP], _I),
    "qmlp_shard_combine": ([_VP, _VP, _I, _I, _VP, _VP], _I),
    "qmlp_shard_info": ([_VP, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I)], _I),
    "qmlp_decode_ctas": ([_VP], _I),
    "qmlp_moe_create": ([ctypes.POINTER(_VP), ctypes.POINTER(qmlp_moe_desc), _VP], _I),
    "qmlp_moe_destroy": ([_VP], None),
    "qmlp_moe_m1_forward": ([_VP, _VP, _I, _VP, _VP, _I, _VP, _VP], _I),
    "qmlp_moe_debug_stages": ([_VP, _VP, _I, _VP, _VP, _I, _VP, _VP, _VP, _VP, _VP], _I),
    "qmlp_moe_check": ([_VP, _VP], _I),
    "qmlp_moe_reserve": ([_VP, _I, _VP], _I),
    "qmlp_moe_forward": ([_VP, _VP, _I, _VP, _VP, _I, _I, _VP, _VP], _I),
    "qmlp_moe_m1_forward_noalloc": ([ctypes.POINTER(qmlp_moe_desc), _VP, _I, _VP, _VP, _I, _VP, _VP], _I),
    "qmlp_lora_create": ([ctypes.POINTER(_VP), _VP, _I, _I, _VP], _I),
    "qmlp_lora_destroy": ([_VP], None),
    "qmlp_lora_set": ([_VP, _I, ctypes.POINTER(qmlp_adapter), _VP], _I),
    "qmlp_lora_forward": ([_VP, _VP, _VP, _I, _VP, _VP], _I),
    "qmlp_train_create": ([ctypes.POINTER(_VP), _VP, _I, _VP], _I),
    "qmlp_train_destroy": ([_VP], None),
    "qmlp_train_saved_bytes": ([_VP, _I], ctypes.c_size_t),
    "qmlp_train_forward": ([_VP, ctypes.POINTER(qmlp_adapter), _VP, _I, _VP, _VP, _VP], _I),
    "qmlp_train_backward": ([_VP, ctypes.POINTER(qmlp_adapter), _VP, _I, _VP, _VP, _VP,
                             ctypes.POINTER(qmlp_adapter), _VP], _I),
    "qmlp_adamw_create": ([ctypes.POINTER(_VP), ctypes.POINTER(qmlp_adamw_tensor), _I, _I, _I, _I, _VP], _I),
    "qmlp_adamw_destroy": ([_VP], None),
    "qmlp_adamw_step": ([_VP, ctypes.POINTER(qmlp_adamw_hyper), _VP], _I),
    "qmlp_status_str": ([_I], ctypes.c_char_p),
    "qmlp_abi_version": ([], _I),
}


def lib(path: str | None = None):
    """Load libqmlp.so (raises QmlpError-compatible RuntimeError if absent).
    QMLP_LIB in the environment names another build of it to load instead
    (the index-checking build, lib/libqmlp_bounds.so)."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or os.environ.get("QMLP_LIB") or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"libqmlp.so not built ({p}); run weight_quantized_swiglu_gb300.build.build()")
            L = ctypes.CDLL(p)
            for name, (args, res) in _SIGS.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


_current_stream = None  # torch's current stream as a raw handle, of the current device


def _find_current_stream():
    import torch
    raw, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is not None and dev is not None:  # without the Stream object: 0.16 us, 3.0 with it
        torch.cuda.init()
        return lambda: raw(dev())
    return lambda: torch.cuda.current_stream().cuda_stream


def _stream(s) -> int | None:
    if s is None:
        global _current_stream
        if _current_stream is None:
            _current_stream = _find_current_stream()
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _chk(st: int, where: str):
    if st != QMLP_OK:
        raise QmlpError(st, where)


# ---- C-named thin wrappers --------------------------------------------------
def qmlp_status_str(st: int) -> str:
    return lib().qmlp_status_str(st).decode()


def qmlp_abi_version() -> int:
    return lib().qmlp_abi_version()


def qmlp_create(desc: qmlp_desc, stream=None) -> int:
    h = ctypes.c_void_p()
    st = lib().qmlp_create(ctypes.byref(h), ctypes.byref(desc), _stream(stream))
    _chk(st, "qmlp_create")
    return h.value


def qmlp_destroy(h: int):
    lib().qmlp_destroy(h)


def qmlp_forward(h, x, M, out, stream=None) -> int:
    return lib().qmlp_forward(h, _ptr(x), M, _ptr(out), _stream(stream))


def qmlp_forward_path(h, path, x, M, out, stream=None) -> int:
    return lib().qmlp_forward_path(h, path, _ptr(x), M, _ptr(out), _stream(stream))


def qmlp_forward_stage(h, stage, path, x, M, out, stream=None) -> int:
    return lib().qmlp_forward_stage(h, stage, path, _ptr(x), M, _ptr(out), _stream(stream))


def qmlp_forward_host(h, x_host, M, out_host, stream=None) -> int:
    return lib().qmlp_forward_host(h, _ptr(x_host), M, _ptr(out_host), _stream(stream))


def qmlp_forward_debug(h, path, x, M, act, out, stream=None) -> int:
    return lib().qmlp_forward_debug(h, path, _ptr(x), M, _ptr(act), _ptr(out), _stream(stream))


def qmlp_debug_project(h, which, path, x, M, y, stream=None) -> int:
    return lib().qmlp_debug_project(h, which, path, _ptr(x), M, _ptr(y), _stream(stream))


def qmlp_check(h, stream=None) -> int:
    return lib().qmlp_check(h, _stream(stream))


def qmlp_debug_split(h, x, act_in, M, g, u, out_f32, stream=None) -> int:
    return lib().qmlp_debug_split(h, _ptr(x), _ptr(act_in), M, _ptr(g), _ptr(u), _ptr(out_f32), _stream(stream))


def qmlp_debug_set_wait(h, limit_ns: int, withhold_last_step: bool) -> int:
    return lib().qmlp_debug_set_wait(h, limit_ns, 1 if withhold_last_step else 0)


def qmlp_debug_bounds_enabled() -> int:
    return lib().qmlp_debug_bounds_enabled()


def qmlp_debug_bounds():
    """(status, site, index) of the first failed index check since the last
    call (a checking build; see include/qmlp.h)."""
    site, index = ctypes.c_int(0), ctypes.c_ulonglong(0)
    st = lib().qmlp_debug_bounds(ctypes.byref(site), ctypes.byref(index))
    return st, site.value, index.value


def qmlp_debug_bounds_limit(h, gate_up_bank_bytes: int) -> int:
    return lib().qmlp_debug_bounds_limit(h, gate_up_bank_bytes)


def qmlp_create_shard(desc: qmlp_desc, rank: int, nranks: int, stream=None) -> int:
    h = ctypes.c_void_p()
    st = lib().qmlp_create_shard(ctypes.byref(h), ctypes.byref(desc), rank, nranks, _stream(stream))
    _chk(st, "qmlp_create_shard")
    return h.value


def qmlp_forward_partial(h, x, M, partial, stream=None) -> int:
    return lib().qmlp_forward_partial(h, _ptr(x), M, _ptr(partial), _stream(stream))


def qmlp_shard_combine(h, partials, nranks, M, out, stream=None) -> int:
    return lib().qmlp_shard_combine(h, _ptr(partials), nranks, M, _ptr(out), _stream(stream))


def qmlp_shard_info(h):
    """(rank, nranks, I of the handle)"""
    r, n, i = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    if not lib().qmlp_shard_info(h, ctypes.byref(r), ctypes.byref(n), ctypes.byref(i)):
        raise QmlpError(1, "qmlp_shard_info")
    return r.value, n.value, i.value


def qmlp_decode_ctas(h) -> int:
    return lib().qmlp_decode_ctas(h)


def qmlp_moe_create(desc: qmlp_moe_desc, stream=None) -> int:
    h = ctypes.c_void_p()
    st = lib().qmlp_moe_create(ctypes.byref(h), ctypes.byref(desc), _stream(stream))
    _chk(st, "qmlp_moe_create")
    return h.value


def qmlp_moe_destroy(h: int):
    lib().qmlp_moe_destroy(h)


def qmlp_moe_m1_forward(h, x, xdt, ids, rw, topk, out, stream=None) -> int:
    return lib().qmlp_moe_m1_forward(h, _ptr(x), xdt, _ptr(ids), _ptr(rw), topk, _ptr(out), _stream(stream))


def qmlp_moe_debug_stages(h, x, xdt, ids, rw, topk, out, gu, act, y, stream=None) -> int:
    return lib().qmlp_moe_debug_stages(h, _ptr(x), xdt, _ptr(ids), _ptr(rw), topk, _ptr(out), _ptr(gu),
                                       _ptr(act), _ptr(y), _stream(stream))


def qmlp_moe_reserve(h, max_tokens, stream=None) -> int:
    return lib().qmlp_moe_reserve(h, max_tokens, _stream(stream))


def qmlp_moe_forward(h, x, xdt, ids, rw, topk, M, out, stream=None) -> int:
    return lib().qmlp_moe_forward(h, _ptr(x), xdt, _ptr(ids), _ptr(rw), topk, M, _ptr(out), _stream(stream))


def qmlp_moe_check(h, stream=None) -> int:
    return lib().qmlp_moe_check(h, _stream(stream))


def qmlp_moe_m1_forward_noalloc(banks: qmlp_moe_desc, x, xdt, ids, rw, topk, out, stream=None) -> int:
    """Routed-expert step on caller-owned device banks; allocates nothing."""
    return lib().qmlp_moe_m1_forward_noalloc(ctypes.byref(banks), _ptr(x), xdt, _ptr(ids), _ptr(rw), topk,
                                             _ptr(out), _stream(stream))


def qmlp_lora_create(h, slots, max_rank, stream=None) -> int:
    p = ctypes.c_void_p()
    st = lib().qmlp_lora_create(ctypes.byref(p), h, slots, max_rank, _stream(stream))
    _chk(st, "qmlp_lora_create")
    return p.value


def qmlp_lora_destroy(p: int):
    lib().qmlp_lora_destroy(p)


def qmlp_lora_set(p, slot, adapter: qmlp_adapter | None, stream=None) -> int:
    return lib().qmlp_lora_set(p, slot, None if adapter is None else ctypes.byref(adapter), _stream(stream))


def qmlp_lora_forward(p, x, ids, M, out, stream=None) -> int:
    return lib().qmlp_lora_forward(p, _ptr(x), _ptr(ids), M, _ptr(out), _stream(stream))


def qmlp_train_create(h, max_rank, stream=None) -> int:
    p = ctypes.c_void_p()
    st = lib().qmlp_train_create(ctypes.byref(p), h, max_rank, _stream(stream))
    _chk(st, "qmlp_train_create")
    return p.value


def qmlp_train_destroy(p: int):
    lib().qmlp_train_destroy(p)


def qmlp_train_saved_bytes(p, M) -> int:
    return lib().qmlp_train_saved_bytes(p, M)


def _ref(c):
    return None if c is None else ctypes.byref(c)


def qmlp_train_forward(p, adapter, x, M, out, saved, stream=None) -> int:
    return lib().qmlp_train_forward(p, _ref(adapter), _ptr(x), M, _ptr(out), _ptr(saved), _stream(stream))


def qmlp_train_backward(p, adapter, x, M, saved, dout, dx, grads, stream=None) -> int:
    return lib().qmlp_train_backward(p, _ref(adapter), _ptr(x), M, _ptr(saved), _ptr(dout), _ptr(dx), _ref(grads),
                                     _stream(stream))


def qmlp_adamw_create(tensors, pdt, gdt, state, stream=None) -> int:
    """tensors: a sequence of qmlp_adamw_tensor."""
    h = ctypes.c_void_p()
    arr = (qmlp_adamw_tensor * len(tensors))(*tensors)
    st = lib().qmlp_adamw_create(ctypes.byref(h), arr, len(tensors), pdt, gdt, state, _stream(stream))
    _chk(st, "qmlp_adamw_create")
    return h.value


def qmlp_adamw_destroy(h: int):
    lib().qmlp_adamw_destroy(h)


def qmlp_adamw_step(h, hyper: qmlp_adamw_hyper, stream=None) -> int:
    return lib().qmlp_adamw_step(h, ctypes.byref(hyper), _stream(stream))


# ---- convenience handles ------------------------------------------------------
def _host_or_dev(a):
    """Keep numpy arrays (host) alive and return (address, owner)."""
    if isinstance(a, np.ndarray):
        a = np.ascontiguousarray(a)
        return a.ctypes.data, a
    return _ptr(a), a


class QuantMLP:
    """Dense weight-quantized SwiGLU MLP handle (NVFP4 or FP8 per-channel).

    Weights may be numpy arrays (host) or torch CUDA tensors; they are copied
    into handle-owned device memory at construction."""

    def __init__(self, fmt: str, K: int, I: int, max_M: int, gate, up, down, stream=None, shard=None):
        """shard = (rank, nranks): this rank's tensor-parallel shard of the
        whole layer described by the arguments (qmlp_create_shard)."""
        self.fmt = FMT_NVFP4 if fmt == "nvfp4" else FMT_FP8_PC
        self.K, self.I, self.max_M = K, I, max_M
        keep = []
        projs = []
        for p in (gate, up, down):
            w, o1 = _host_or_dev(p.w)
            s, o2 = _host_or_dev(p.scale)
            keep += [o1, o2]
            projs.append(qmlp_proj(w, s, float(p.global_scale)))
        d = qmlp_desc(self.fmt, K, I, max_M, *projs)
        if shard is None:
            self.h = qmlp_create(d, stream)
        else:
            self.h = qmlp_create_shard(d, shard[0], shard[1], stream)
            self.I = I // shard[1]
        self.rank, self.nranks, _ = qmlp_shard_info(self.h)

    @classmethod
    def from_case(cls, case, max_M=None, stream=None, shard=None):
        return cls(case.fmt, case.K, case.I, max_M or case.M, case.gate, case.up, case.down, stream, shard)

    def forward_partial(self, x, partial, M=None, stream=None):
        """fp32 [M, K] partial of a tensor-parallel shard (no down factor)."""
        M = x.shape[0] if M is None else M
        _chk(qmlp_forward_partial(self.h, x, M, partial, stream), "qmlp_forward_partial")
        return partial

    def combine(self, partials, out, M=None, stream=None):
        """out = bf16(sigma_d * rank-ordered sum of partials [nranks, M, K])."""
        M = partials.shape[1] if M is None else M
        _chk(qmlp_shard_combine(self.h, partials, self.nranks, M, out, stream), "qmlp_shard_combine")
        return out

    def debug_split(self, x, act_in, g, u, out_f32, M=None, stream=None):
        M = x.shape[0] if M is None else M
        _chk(qmlp_debug_split(self.h, x, act_in, M, g, u, out_f32, stream), "qmlp_debug_split")

    def set_wait(self, limit_ns: int, withhold_last_step: bool = False):
        _chk(qmlp_debug_set_wait(self.h, limit_ns, withhold_last_step), "qmlp_debug_set_wait")

    def bounds_limit(self, gate_up_bank_bytes: int):
        _chk(qmlp_debug_bounds_limit(self.h, gate_up_bank_bytes), "qmlp_debug_bounds_limit")

    def forward(self, x, out, M=None, path=PATH_AUTO, stream=None):
        M = x.shape[0] if M is None else M
        _chk(qmlp_forward_path(self.h, path, x, M, out, stream), "qmlp_forward")
        return out

    def forward_stage(self, stage, x, out, M, path=PATH_AUTO, stream=None):
        _chk(qmlp_forward_stage(self.h, stage, path, x, M, out, stream), "qmlp_forward_stage")

    def forward_debug(self, x, act, out, M=None, path=PATH_AUTO, stream=None):
        M = x.shape[0] if M is None else M
        _chk(qmlp_forward_debug(self.h, path, x, M, act, out, stream), "qmlp_forward_debug")
        return act, out

    def forward_host(self, x_host, out_host, M=None, stream=None):
        M = x_host.shape[0] if M is None else M
        _chk(qmlp_forward_host(self.h, x_host, M, out_host, stream), "qmlp_forward_host")
        return out_host

    def debug_project(self, which, x, y, M=None, path=PATH_AUTO, stream=None):
        M = x.shape[0] if M is None else M
        _chk(qmlp_debug_project(self.h, which, path, x, M, y, stream), "qmlp_debug_project")
        return y

    def check(self, stream=None):
        _chk(qmlp_check(self.h, stream), "qmlp_check")

    def decode_ctas(self):
        """CTAs of the I-partitioned single-launch decode kernel (0: not used)."""
        return qmlp_decode_ctas(self.h)

    def close(self):
        if getattr(self, "h", None):
            qmlp_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MoeAWQ:
    """Routed-expert AWQ int4 g32 handle (one token; M tokens after reserve())."""

    def __init__(self, E, K, I, meta_bytes, w13, w13_meta, w2, w2_meta, stream=None):
        self.E, self.K, self.I, self.meta = E, K, I, meta_bytes
        ptrs = [_host_or_dev(a) for a in (w13, w13_meta, w2, w2_meta)]
        d = qmlp_moe_desc(E, K, I, meta_bytes, *[p for p, _ in ptrs])
        self.h = qmlp_moe_create(d, stream)

    @classmethod
    def from_case(cls, case, meta_bytes=4, stream=None):
        m13 = case.w13_meta4 if meta_bytes == 4 else case.w13_meta3
        m2 = case.w2_meta4 if meta_bytes == 4 else case.w2_meta3
        return cls(case.E, case.K, case.I, meta_bytes, case.w13, m13, case.w2, m2, stream)

    def forward(self, x, xdt, ids, rw, out, topk=None, stream=None):
        topk = ids.shape[0] if topk is None else topk
        _chk(qmlp_moe_m1_forward(self.h, x, xdt, ids, rw, topk, out, stream), "qmlp_moe_m1_forward")
        return out

    def reserve(self, max_tokens, stream=None):
        _chk(qmlp_moe_reserve(self.h, max_tokens, stream), "qmlp_moe_reserve")

    def forward_tokens(self, x, xdt, ids, rw, out, stream=None):
        """M tokens: x [M, K], ids / rw [M, topk], out [M, K]."""
        M, topk = ids.shape
        _chk(qmlp_moe_forward(self.h, x, xdt, ids, rw, topk, M, out, stream), "qmlp_moe_forward")
        return out

    def debug_stages(self, x, xdt, ids, rw, out, gu=None, act=None, y=None, topk=None, stream=None):
        topk = ids.shape[0] if topk is None else topk
        _chk(qmlp_moe_debug_stages(self.h, x, xdt, ids, rw, topk, out, gu, act, y, stream),
             "qmlp_moe_debug_stages")

    def check(self, stream=None):
        _chk(qmlp_moe_check(self.h, stream), "qmlp_moe_check")

    def close(self):
        if getattr(self, "h", None):
            qmlp_moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _device_buffer(who, name, t, nbytes):
    """Refuse a tensor that a kernel would read or write past its end, or not
    in the order of its elements."""
    if not t.is_cuda or not t.is_contiguous() or t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{who}: {name} has to be a contiguous CUDA tensor of {nbytes} bytes or more")


def _device_rows(who, M, K, **tensors):
    """Refuse what is not M rows of K 16-bit values on the device (raw addresses
    are the caller's)."""
    for name, t in tensors.items():
        if isinstance(t, int):
            continue
        _device_buffer(who, name, t, 2 * M * K)
        if t.dim() > 1 and t.shape[-1] * t.element_size() != 2 * K:
            raise ValueError(f"{who}: {name} has rows of {t.shape[-1]} values, {K} are wanted")


class Adapter:
    """A low-rank adapter of the block: scale (alpha / r) and, for each adapted
    projection, A [r, in] and B [out, r], contiguous bf16 CUDA tensors of one
    rank. A projection that is not adapted has neither."""

    def __init__(self, scale, gate_a=None, gate_b=None, up_a=None, up_b=None, down_a=None, down_b=None):
        import torch
        self.parts = dict(zip(ADAPTER_PARTS, (gate_a, gate_b, up_a, up_b, down_a, down_b)))
        self.scale, self.rank = float(scale), 0
        for n, t in self.parts.items():
            if t is None:
                continue
            if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 2 or not t.is_contiguous():
                raise ValueError(f"Adapter: {n} has to be a contiguous bf16 CUDA matrix")
            r = t.shape[0] if n.endswith("_a") else t.shape[1]
            if self.rank not in (0, r):
                raise ValueError(f"Adapter: {n} has rank {r}, another part {self.rank}")
            self.rank = r
        for p in ("gate", "up", "down"):
            if (self.parts[p + "_a"] is None) != (self.parts[p + "_b"] is None):
                raise ValueError(f"Adapter: {p} needs both A and B")
        self.c = qmlp_adapter(self.rank, self.scale, *[_ptr(t) for t in self.parts.values()])

    def check(self, K, I):
        want = {"gate": (I, K), "up": (I, K), "down": (K, I)}
        for n, t in self.parts.items():
            if t is not None:
                out, inp = want[n[:-2]]
                shape = (self.rank, inp) if n.endswith("_a") else (out, self.rank)
                if tuple(t.shape) != shape:
                    raise ValueError(f"Adapter: {n} is {tuple(t.shape)}, {shape} is wanted")


class LoraMLP:
    """A QuantMLP with `slots` low-rank adapters, one a token (qmlp_lora_*).
    The QuantMLP has to stay open while this object is."""

    def __init__(self, mlp: QuantMLP, slots: int, max_rank: int, stream=None):
        self.mlp, self.slots = mlp, slots
        self.h = qmlp_lora_create(mlp.h, slots, max_rank, stream)

    def set(self, slot, adapter: Adapter | None, stream=None):
        """Copy an adapter into a slot (None: empty it), in stream order."""
        if adapter is not None:
            adapter.check(self.mlp.K, self.mlp.I)
        _chk(qmlp_lora_set(self.h, slot, None if adapter is None else adapter.c, stream), "qmlp_lora_set")

    def forward(self, x, ids, out, M=None, stream=None):
        """x [M, K] bf16, ids [M] int32 (the token's slot; none: -1), out [M, K] bf16."""
        M = x.shape[0] if M is None else M
        _device_rows("LoraMLP", M, self.mlp.K, x=x, out=out)
        if not isinstance(ids, int) and (not ids.is_cuda or ids.element_size() != 4 or ids.is_floating_point() or
                                         not ids.is_contiguous() or ids.numel() < M):
            raise ValueError(f"LoraMLP: ids has to be a contiguous int32 CUDA tensor of {M} values")
        _chk(qmlp_lora_forward(self.h, x, ids, M, out, stream), "qmlp_lora_forward")
        return out

    def close(self):
        if getattr(self, "h", None):
            qmlp_lora_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class TrainMLP:
    """Forward and backward of a QuantMLP with frozen weights and one low-rank
    adapter or none (qmlp_train_*). The QuantMLP has to stay open while this
    object is."""

    def __init__(self, mlp: QuantMLP, max_rank: int, stream=None):
        self.mlp = mlp
        self.h = qmlp_train_create(mlp.h, max_rank, stream)

    def saved_bytes(self, M):
        """Bytes of the buffer that forward fills for backward."""
        return qmlp_train_saved_bytes(self.h, M)

    def _adapter(self, a):
        if a is None:
            return None
        a.check(self.mlp.K, self.mlp.I)
        return a.c

    def _saved(self, saved, M):
        if not isinstance(saved, int):
            _device_buffer("TrainMLP", "saved", saved, self.saved_bytes(M))

    def forward(self, x, out, saved, adapter: Adapter | None = None, M=None, stream=None):
        """x, out [M, K] bf16; saved: saved_bytes(M) bytes on the device or more
        (a buffer for the longest batch serves the shorter ones)."""
        M = x.shape[0] if M is None else M
        self._saved(saved, M)
        _device_rows("TrainMLP", M, self.mlp.K, x=x, out=out)
        _chk(qmlp_train_forward(self.h, self._adapter(adapter), x, M, out, saved, stream), "qmlp_train_forward")
        return out

    def backward(self, x, saved, dout, dx, adapter: Adapter | None = None, grads: Adapter | None = None, M=None,
                 stream=None):
        """dout, dx [M, K] bf16; grads: the tensors that take the gradients of
        the adapter's parts (its scale is not used)."""
        M = x.shape[0] if M is None else M
        self._saved(saved, M)
        _device_rows("TrainMLP", M, self.mlp.K, x=x, dout=dout, dx=dx)
        # (an Adapter without parts has no rank: no gradient is wanted)
        if adapter is not None and grads is not None and grads.rank not in (0, adapter.rank):
            raise ValueError(f"TrainMLP: gradients of rank {grads.rank} for an adapter of rank {adapter.rank}")
        _chk(qmlp_train_backward(self.h, self._adapter(adapter), x, M, saved, dout, dx, self._adapter(grads), stream),
             "qmlp_train_backward")
        return dx

    def close(self):
        if getattr(self, "h", None):
            qmlp_train_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class AdamW:
    """AdamW over many CUDA tensors, one launch a step (qmlp_adamw_*).

    params: fp32 or bf16; grads: fp32 or bf16; m, v: fp32, or float8_e4m3fn
    (or uint8) codes with m_scale / v_scale, fp32 [ceil(n / 256)] a tensor
    (v's codes are those of its square root). master: fp32 copies of bf16
    parameters, which the step is then taken on. The lists go tensor by
    tensor; the tensors are contiguous, are kept alive by this object, and
    are updated in place."""

    def __init__(self, params, grads, m, v, m_scale=None, v_scale=None, master=None, stream=None):
        import torch
        count = len(params)
        lists = {"params": params, "grads": grads, "m": m, "v": v, "m_scale": m_scale, "v_scale": v_scale,
                 "master": master}
        for name, ts in lists.items():
            if ts is None:
                continue
            if len(ts) != count:
                raise ValueError(f"AdamW: {len(ts)} tensors in {name}, {count} in params")
            for i, t in enumerate(ts):
                n = params[i].numel()
                want = -(-n // 256) if name.endswith("scale") else n
                if not t.is_cuda or not t.is_contiguous() or t.numel() != want or t.dtype != ts[0].dtype:
                    raise ValueError(f"AdamW: {name}[{i}] has to be a contiguous CUDA tensor of {want} elements, "
                                     f"all of one type")
        if not count:
            raise ValueError("AdamW: no tensors")
        kinds = {torch.float32: DT_FP32, torch.bfloat16: DT_BF16}
        eight = m[0].dtype in (torch.uint8, torch.float8_e4m3fn)
        if (params[0].dtype not in kinds or grads[0].dtype not in kinds or m[0].dtype != v[0].dtype or
                not (eight or m[0].dtype == torch.float32) or eight != (m_scale is not None) or
                eight != (v_scale is not None) or
                any(ts is not None and ts[0].dtype != torch.float32 for ts in (m_scale, v_scale, master))):
            raise ValueError("AdamW: params and grads are fp32 or bf16, states fp32 or 8-bit codes with fp32 scales, "
                             "a master fp32")
        at = lambda ts, i: None if ts is None else ts[i].data_ptr()  # noqa: E731
        ts = [qmlp_adamw_tensor(params[i].numel(), at(params, i), at(master, i), at(grads, i), at(m, i), at(v, i),
                                at(m_scale, i), at(v_scale, i)) for i in range(count)]
        self.h = qmlp_adamw_create(ts, kinds[params[0].dtype], kinds[grads[0].dtype],
                                   STATE_8BIT if eight else STATE_FP32, stream)
        self._keep = lists
        self._step = lib().qmlp_adamw_step

    def step(self, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, grad_scale=1.0, stream=None):
        hyper = qmlp_adamw_hyper(lr, beta1, beta2, eps, weight_decay, grad_scale, step)
        _chk(self._step(self.h, hyper, _stream(stream)), "qmlp_adamw_step")

    def close(self):
        if getattr(self, "h", None):
            qmlp_adamw_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
