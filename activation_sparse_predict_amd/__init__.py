"""Python binding of the C ABI in include/pi.h (libpi.so, HIP for gfx950).

Argument marshalling only: every step of the sparse FFN runs in the library's
HIP kernels.  PyTorch provides device memory and the current stream.  There is
no CPU fallback: if the shared library is missing or fails to load, importing
the binding's entry points raises.

Entry points (same names and meaning as the C functions):
  workspace_bytes(layers, batch)
  predict(layer, x, idx, count, scores=None, mask=None, ws=None)
  sparse_ffn(layer, x, idx, count, y, mask=None, ws=None)
  ffn_stack(layers, x, out, counts=None, trace=None, ws=None, nz_counts=None)
  Cache(k_pool, v_pool, meta, slots, max_pages) with .extend, .append, .fork, .release, .compact, .reserve
  attn_prompt(q, k, v, out, cu)
  attn_decode(cache, layer, q, out, prefix=None, seqs=None)
  Q4Matrix(nibbles, scales, bias, batch) and matvec(mat, x, y)

The last four lines' operators have no gradient and refuse tensors that want one.  Tensors and
handles of a call have to live until its work on the stream is done.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpi.so")

PI_OK, PI_EINVAL, PI_EUNSUPPORTED, PI_EWORKSPACE, PI_EHIP = 0, 1, 2, 3, 4
PI_F32, PI_F16, PI_Q4_0, PI_BF16 = 0, 1, 2, 3
PI_RELU, PI_REGLU, PI_RELU2 = 0, 1, 2

_DTYPE = {"f32": PI_F32, "f16": PI_F16, "q4_0": PI_Q4_0}
_ACT = {"relu": PI_RELU, "reglu": PI_REGLU, "relu2": PI_RELU2}


class PiError(RuntimeError):
    def __init__(self, status: int, where: str):
        detail = f" [{lib().pi_last_hip_error().decode()}]" if status == PI_EHIP else ""
        super().__init__(f"{where}: {status_str(status)} ({status}){detail}")
        self.status = status


class PiMat(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class PiLayer(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("ffn", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("act", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("p_dtype", ctypes.c_int32),
                ("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("pbias", ctypes.c_void_p), ("gate", PiMat), ("up", PiMat), ("downT", PiMat), ("b_down", ctypes.c_void_p),
                ("hot", ctypes.c_int32), ("dense_frac", ctypes.c_float)]


class PiTrace(ctypes.Structure):
    _fields_ = [("x_in", ctypes.c_void_p), ("scores", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("idx", ctypes.c_void_p), ("count", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("events", ctypes.POINTER(ctypes.c_void_p)), ("n_events", ctypes.c_int32)]


class PiHeads(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class PiCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("meta", ctypes.c_void_p),
                ("layers", ctypes.c_int32), ("pages", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("page", ctypes.c_int32), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("slots", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


_HEADS = struct.Struct("@Pqq")                         # PiHeads

# bits of a cache's error word
PI_CACHE_ESLOT, PI_CACHE_EPAGE, PI_CACHE_EFULL, PI_CACHE_ELENGTH, PI_CACHE_EPREFIX = 1, 2, 4, 8, 16


# kernels of one layer, in the order the trace events bracket them
LAYER_KERNELS = {1: ("k_predict_t", "k_score", "k_down"),
                 2: ("k_bglue", "k_bpred1", "k_bsplit_t", "k_bscore", "k_compact", "k_bup", "k_bdown")}


# the layout of the structures above; the library must report the same version
ABI_VERSION = 6

_lib = None


def lib():
    """Load libpi.so (raises if it is not built, or built from another ABI version)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built (run __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        # entry points that are added leave the version as it is: a library without them is an older one
        missing = [name for name in EXPORTED if not hasattr(L, name)]
        got = int(L.pi_abi_version()) if "pi_abi_version" not in missing else None
        if got != ABI_VERSION or missing:
            raise RuntimeError(f"{LIB_PATH} has ABI version {got}, this binding expects {ABI_VERSION}"
                               + (f" and {', '.join(missing)}" if missing else "")
                               + " (rebuild with __graft_entry__.build())")
        L.pi_abi_version.restype = I32
        L.pi_status_str.argtypes = [ctypes.c_int]
        L.pi_status_str.restype = ctypes.c_char_p
        L.pi_workspace_bytes.argtypes = [P, I32, I32]
        L.pi_workspace_bytes.restype = SZ
        L.pi_predict.argtypes = [P, P, I32, P, P, P, P, P, SZ, P]
        L.pi_predict.restype = ctypes.c_int
        L.pi_sparse_ffn.argtypes = [P, P, I32, P, P, P, P, P, SZ, P]
        L.pi_sparse_ffn.restype = ctypes.c_int
        L.pi_ffn_stack.argtypes = [P, I32, P, I32, P, P, P, P, P, SZ, P]
        L.pi_ffn_stack.restype = ctypes.c_int
        L.pi_ffn_stack_static.argtypes = [P, I32, P, I32, P, P, P, P, P]
        L.pi_ffn_stack_static.restype = ctypes.c_int
        L.pi_last_hip_error.restype = ctypes.c_char_p
        F, I64 = ctypes.c_float, ctypes.c_int64
        for name, res, args in (
                ("pi_cache_meta_words", SZ, [I32, I32, I32]),
                ("pi_cache_workspace_bytes", SZ, [P]),
                ("pi_cache_extend", ctypes.c_int, [P, P, P, I32, P]),
                ("pi_cache_append", ctypes.c_int, [P, I32, P, P, I32, P, P, I32, P]),
                ("pi_cache_fork", ctypes.c_int, [P, P, P, I32, P, SZ, P]),
                ("pi_cache_release", ctypes.c_int, [P, P, I32, P]),
                ("pi_cache_compact", ctypes.c_int, [P, P, P, SZ, P]),
                ("pi_attn_prompt", ctypes.c_int, [P, P, P, P, I32, I32, I32, I32, I32, P, I32, F, P]),
                ("pi_attn_workspace_bytes", SZ, [P, I32, I32]),
                ("pi_attn_decode", ctypes.c_int, [P, I32, P, P, I32, I32, P, P, F, P, SZ, P]),
                ("pi_matvec_workspace_bytes", SZ, [I32, I32, I32]),
                ("pi_matvec", ctypes.c_int, [P, I32, I32, P, P, I32, I64, P, I32, I64, I32, P, SZ, P])):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def abi_version() -> int:
    return int(lib().pi_abi_version())


def status_str(s: int) -> str:
    return lib().pi_status_str(int(s)).decode()


def _p(t) -> Optional[int]:
    """Device address of a tensor (or an int address), None for None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_torch = None                                          # an import statement in every call would take its time


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _gpu_of(t) -> Optional[int]:
    """The GPU of a tensor; None for an address, whose caller sees to the current GPU."""
    dev = t.get_device() if hasattr(t, "get_device") else -1
    return dev if dev >= 0 else None


def _stream_on(dev: Optional[int], stream):
    """The handle of a stream, or of the current stream of a GPU."""
    if dev is None:
        return _stream(stream)
    if stream is None:
        return (_torch or _load_torch())._C._cuda_getCurrentRawStream(dev)
    if getattr(stream, "device_index", dev) != dev:
        raise PiError(PI_EINVAL, "stream of another GPU")
    return _stream(stream)


def _stream_of(dev: int, handle: int):
    import torch
    return torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)


def _on(dev: Optional[int], call, *args) -> int:
    """A call of the library with GPU `dev` current (None: as it is).  A kernel goes to the current GPU where its stream's
    handle is 0, which every GPU's default stream has."""
    if dev is None:
        return call(*args)
    gpus = (_torch or _load_torch())._C
    here = gpus._cuda_getDevice()
    if here == dev:
        return call(*args)
    gpus._cuda_setDevice(dev)
    try:
        return call(*args)
    finally:
        gpus._cuda_setDevice(here)


def _check(status: int, where: str):
    if status != PI_OK:
        raise PiError(status, where)


# ------------------------------------------------------------------ layers
class DeviceLayer:
    """One layer's tensors resident on the GPU plus the matching pi_layer record."""

    def __init__(self, *, d, ffn, rank, act, w_dtype, p_dtype, A, B, bias, up, downT, gate=None,
                 b_down=None, pbias=None, hot=0, dense_frac=0.0):
        self.d, self.ffn, self.rank = int(d), int(ffn), int(rank)
        self.hot = int(hot)
        self.dense_frac = float(dense_frac)
        self.act, self.w_dtype, self.p_dtype = act, w_dtype, p_dtype
        self.A, self.B, self.bias, self.up, self.downT, self.gate, self.b_down = \
            A, B, bias, up, downT, gate, b_down
        self.pbias = pbias
        self.struct = self._make_struct()

    @staticmethod
    def _mat(m):
        if m is None:
            return PiMat(None, None)
        if isinstance(m, tuple):            # Q4_0: (nibbles, scales)
            return PiMat(m[0].data_ptr(), m[1].data_ptr())
        return PiMat(m.data_ptr(), None)

    def _make_struct(self) -> PiLayer:
        return PiLayer(self.d, self.ffn, self.rank, _ACT[self.act], _DTYPE[self.w_dtype],
                       _DTYPE[self.p_dtype], _p(self.A), _p(self.B), _p(self.bias),
                       _p(self.pbias), self._mat(self.gate), self._mat(self.up), self._mat(self.downT),
                       _p(self.b_down), self.hot, self.dense_frac)

    @classmethod
    def upload(cls, lw, device="cuda") -> "DeviceLayer":
        """Copy a host layer (numpy arrays; Q4_0 matrices with .nibbles/.scales) to the GPU."""
        import numpy as np
        import torch

        def t(a):
            if a is None:
                return None
            if hasattr(a, "nibbles"):
                nib = torch.from_numpy(np.ascontiguousarray(a.nibbles)).to(device)
                sc = torch.from_numpy(np.ascontiguousarray(a.scales).view(np.int16)).to(device)
                return (nib, sc)
            return torch.from_numpy(np.ascontiguousarray(a)).to(device)

        cfg = lw.cfg
        return cls(d=cfg.d, ffn=cfg.ffn, rank=cfg.rank, act=cfg.act, w_dtype=cfg.w_dtype,
                   p_dtype=cfg.p_dtype, A=t(lw.A), B=t(lw.B), bias=t(lw.bias), up=t(lw.up),
                   downT=t(lw.downT), gate=t(lw.gate), b_down=t(lw.b_down),
                   pbias=t(getattr(lw, "pbias", None)), hot=int(getattr(lw, "hot", 0) or 0),
                   dense_frac=float(getattr(lw, "dense_frac", 0.0) or 0.0))

    def nbytes(self) -> int:
        tot = 0
        for m in (self.A, self.B, self.bias, self.pbias, self.up, self.downT, self.gate, self.b_down):
            if m is None:
                continue
            for x in (m if isinstance(m, tuple) else (m,)):
                tot += x.numel() * x.element_size()
        return tot


def _layer_array(layers: Sequence[DeviceLayer]):
    arr = (PiLayer * len(layers))()
    for i, L in enumerate(layers):
        arr[i] = L.struct
    return arr


# ------------------------------------------------------------- entry points
def workspace_bytes(layers, batch: int = 1) -> int:
    layers = [layers] if isinstance(layers, DeviceLayer) else list(layers)
    arr = _layer_array(layers)
    return int(lib().pi_workspace_bytes(ctypes.cast(arr, ctypes.c_void_p), len(layers), batch))


def alloc_workspace(layers, batch: int = 1, device=None):
    """A workspace on `device`: unless it is given, where the first layer lies."""
    import torch
    layers = [layers] if isinstance(layers, DeviceLayer) else list(layers)
    n = workspace_bytes(layers, batch)
    if n == 0:
        raise PiError(PI_EINVAL, "workspace_bytes")
    if device is None:
        gpu = _gpu_of(layers[0].A)
        device = "cuda" if gpu is None else torch.device("cuda", gpu)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _call_workspace(layers, batch: int, dev: Optional[int], stream):
    """A workspace of one call.  It is given back when the call returns, before its work is done, so it is memory of the
    call's own stream: the next to get it there comes after that work."""
    if dev is None or stream is None:
        return alloc_workspace(layers, batch)
    import torch
    with torch.cuda.stream(_stream_of(dev, _stream_on(dev, stream))):
        return alloc_workspace(layers, batch)


def predict(layer: DeviceLayer, x, idx, count, scores=None, mask=None, ws=None, batch: int = 1,
            stream=None):
    dev = _gpu_of(x)
    ws = _call_workspace(layer, batch, dev, stream) if ws is None else ws
    st = _on(dev, lib().pi_predict, ctypes.byref(layer.struct), _p(x), batch, _p(scores), _p(mask), _p(idx),
             _p(count), _p(ws), ws.numel(), _stream_on(dev, stream))
    _check(st, "pi_predict")


def sparse_ffn(layer: DeviceLayer, x, idx, count, y, mask=None, ws=None, batch: int = 1,
               stream=None):
    dev = _gpu_of(x)
    ws = _call_workspace(layer, batch, dev, stream) if ws is None else ws
    st = _on(dev, lib().pi_sparse_ffn, ctypes.byref(layer.struct), _p(x), batch, _p(idx), _p(count),
             _p(mask), _p(y), _p(ws), ws.numel(), _stream_on(dev, stream))
    _check(st, "pi_sparse_ffn")


def make_trace(n_layers: int, recs: Sequence[dict]):
    """Trace records; a record's optional "events" entry is a list of hipEvent_t handles
    (ints, e.g. from HipEvents) or objects with a .cuda_event handle."""
    arr = (PiTrace * n_layers)()
    keep = []
    for i, r in enumerate(recs):
        evs = r.get("events")
        if evs:
            ptrs = (ctypes.c_void_p * len(evs))(*[e if isinstance(e, int) else e.cuda_event for e in evs])
            keep.append(ptrs)
            ev_arg, n_ev = ctypes.cast(ptrs, ctypes.POINTER(ctypes.c_void_p)), len(evs)
        else:
            ev_arg, n_ev = None, 0
        arr[i] = PiTrace(_p(r.get("x_in")), _p(r.get("scores")), _p(r.get("mask")),
                         _p(r.get("idx")), _p(r.get("count")), _p(r.get("y")), ev_arg, n_ev)
    arr._keep = keep
    return arr


class Stack:
    """A stack of DeviceLayers with its layer array and workspace kept alive."""

    def __init__(self, layers: Sequence[DeviceLayer], batch: int = 1, ws=None):
        self.layers = list(layers)
        self.batch = batch
        self.arr = _layer_array(self.layers)
        self.ws = alloc_workspace(self.layers, batch) if ws is None else ws

    def __call__(self, x, out, counts=None, trace=None, stream=None, nz_counts=None):
        tr = None if trace is None else ctypes.cast(trace, ctypes.c_void_p)
        dev = _gpu_of(x)
        st = _on(dev, lib().pi_ffn_stack, ctypes.cast(self.arr, ctypes.c_void_p), len(self.layers), _p(x),
                 self.batch, _p(out), _p(counts), _p(nz_counts), tr, _p(self.ws),
                 self.ws.numel(), _stream_on(dev, stream))
        _check(st, "pi_ffn_stack")


def ffn_stack(layers, x, out, counts=None, trace=None, ws=None, batch: int = 1, stream=None, nz_counts=None):
    layers = list(layers)
    ws = _call_workspace(layers, batch, _gpu_of(x), stream) if ws is None else ws
    Stack(layers, batch, ws)(x, out, counts, trace, stream, nz_counts)


STATIC_WORKSPACE_BYTES = 96 << 20   # PI_STATIC_WORKSPACE_BYTES


def ffn_stack_static(layers, x, out, counts=None, trace=None, batch: int = 1, stream=None, nz_counts=None):
    """pi_ffn_stack_static: the stack on the library's own per-GPU scratch array (no workspace)."""
    arr = _layer_array(list(layers))
    tr = None if trace is None else ctypes.cast(trace, ctypes.c_void_p)
    dev = _gpu_of(x)
    st = _on(dev, lib().pi_ffn_stack_static, ctypes.cast(arr, ctypes.c_void_p), len(arr), _p(x), batch, _p(out),
             _p(counts), _p(nz_counts), tr, _stream_on(dev, stream))
    _check(st, "pi_ffn_stack_static")


# ------------------------------------------ the attention half of a decoder layer
# A call on a few tokens takes the GPU less time than its checks take the host, so these are kept short:
# each attribute of a tensor is asked for once, and the current stream without an object for it.
_KINDS = None


def _torch_names():
    global _KINDS
    import torch
    _KINDS = {torch.float32: PI_F32, torch.float16: PI_F16, torch.bfloat16: PI_BF16, torch.int32: "int32"}
    return _KINDS


def _dtype_of(t) -> int:
    """pi_dtype of a float tensor (other types: PI_EINVAL)."""
    kind = (_KINDS or _torch_names()).get(t.dtype)
    if kind is None or kind == "int32":
        raise PiError(PI_EINVAL, f"tensor of {t.dtype}")
    return kind


def _need(ok: bool, what: str):
    if not ok:
        raise PiError(PI_EINVAL, what)


def _gpu(what: str, first, *tensors) -> int:
    """The GPU on which all tensors (None aside) lie: a kernel cannot follow an address of the host's.  None of them may want
    a gradient, which these operators do not have."""
    dev = first.get_device()
    for t in tensors:
        if t is not None:
            if t.get_device() != dev:
                raise PiError(PI_EINVAL, what)
            if t.requires_grad and (_torch or _load_torch()).is_grad_enabled():
                raise PiError(PI_EINVAL, what.split(":")[0]
                              + ": a tensor wants a gradient (torch.no_grad says that none is wanted)")
    if dev < 0:
        raise PiError(PI_EINVAL, what)
    return dev


def _ints(t, n: Optional[int], what: str) -> Optional[int]:
    """Address of a contiguous int32 tensor of n elements (any number where n is None), or None for None."""
    if t is None:
        return None
    shape = t.shape
    if len(shape) != 1 or (n is not None and shape[0] != n) or not t.is_contiguous() \
            or (_KINDS or _torch_names()).get(t.dtype) != "int32":
        raise PiError(PI_EINVAL, what)
    return t.data_ptr()


def _heads(t, shape, what: str) -> bytes:
    """The pi_heads of a [tokens][heads][dim] tensor with strides, the last dimension contiguous, as the bytes of the
    structure (which take a third of a PiHeads object's time)."""
    token, head, one = t.stride()
    if one != 1 and shape[2] != 1:
        raise PiError(PI_EINVAL, what)
    # the stride of a dimension of one element says nothing
    return _HEADS.pack(t.data_ptr(), token if shape[0] > 1 else 0, head if shape[1] > 1 else 0)


def _capturing(dev: int, handle: Optional[int] = None) -> bool:
    """Whether a graph is being captured on a stream, or on the current one."""
    import torch
    if handle is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(_stream_of(dev, handle)):
        return torch.cuda.is_current_stream_capturing()


def _mark(dev: int):
    """An event behind the work of a GPU's current stream so far."""
    import torch
    if _capturing(dev):                                # what is captured runs after all that came before it
        return None
    stream = torch.cuda.current_stream(dev)
    return stream.record_event()


def _wait_for(dev: int, handle: int, event) -> bool:
    """A stream waits for an event; False inside a capture, which cannot wait for what is outside of it."""
    if _capturing(dev, handle):
        return False
    _stream_of(dev, handle).wait_event(event)
    return True


class _Scratch:
    """Workspace memory that a handle keeps for its calls.

    Torch gives out memory again when the work that uses it is on its way on the stream it was taken on, so that stream may
    still be reading what another stream's call would write: such a stream waits, once, for the work there was when the
    memory was taken.  (A capture begins when the work before it is done; torch.cuda.graph sees to that.)"""

    def __init__(self, n: int, device):
        import torch
        self.mem = torch.empty(n, dtype=torch.uint8, device=device)
        self.dev, self.address, self.bytes = self.mem.get_device(), self.mem.data_ptr(), n
        self.streams, self.taken = {torch._C._cuda_getCurrentRawStream(self.dev)}, _mark(self.dev)

    def on(self, handle: int) -> int:
        """Its address, for a call on a stream."""
        if handle not in self.streams and (self.taken is None or _wait_for(self.dev, handle, self.taken)):
            self.streams.add(handle)
        return self.address


class Cache:
    """A paged key/value cache (pi_cache in include/pi.h) over tensors of the caller's.

    k_pool, v_pool: [layers][pages][kv_heads][page][dim], float16 or bfloat16.  meta: the page
    tables, one int32 tensor; .table, .lens, .ref, .free and .words are views of its parts.
    The workspace of attn_decode is one buffer that grows when a call needs more, never inside a
    capture: a call that is captured has to have run once before with the same sizes, or .reserve
    has been called.  Calls on one cache belong on one stream."""

    def __init__(self, k_pool, v_pool, meta, slots: int, max_pages: int):
        import torch
        _need(k_pool.dim() == 5 and k_pool.shape == v_pool.shape and k_pool.dtype == v_pool.dtype
              and k_pool.is_contiguous() and v_pool.is_contiguous(), "Cache: pools")
        layers, pages, kv_heads, page, dim = k_pool.shape
        self.k_pool, self.v_pool, self.meta = k_pool, v_pool, meta
        self.layers, self.pages, self.kv_heads, self.page, self.dim = layers, pages, kv_heads, page, dim
        self.slots, self.max_pages = int(slots), int(max_pages)
        words = self.meta_words(slots, max_pages, pages)
        _need(words > 0 and meta.dtype == torch.int32 and meta.dim() == 1 and meta.is_contiguous()
              and meta.numel() == words, "Cache: meta")
        _gpu("Cache: tensors of one GPU", k_pool, v_pool, meta)
        self.struct = PiCache(_p(k_pool), _p(v_pool), _p(meta), layers, pages, kv_heads, page, dim,
                              _dtype_of(k_pool), self.slots, self.max_pages)
        self._ref = ctypes.byref(self.struct)
        a = self.slots * self.max_pages
        b = a + self.slots
        self.table, self.lens = meta[:a].view(self.slots, self.max_pages), meta[a:b]
        self.ref, self.free = meta[b:b + pages], meta[b + pages:b + 2 * pages]
        self.words = meta[b + 2 * pages:]
        n = int(lib().pi_cache_workspace_bytes(self._ref))
        if n == 0:                                   # say which rule it is
            _check(lib().pi_cache_release(self._ref, None, 1, None), "Cache")
        self.dtype, self._lib = k_pool.dtype, lib()
        self._ws = _Scratch(n, k_pool.device)
        self.ws = self._ws.mem
        self._attn_need, self._attn_ws, self._attn_before = {}, None, []

    @staticmethod
    def meta_words(slots: int, max_pages: int, pages: int) -> int:
        return int(lib().pi_cache_meta_words(slots, max_pages, pages))

    @classmethod
    def create(cls, layers: int, pages: int, kv_heads: int, page: int, dim: int, slots: int, max_pages: int,
               dtype=None, device="cuda") -> "Cache":
        """An empty cache in tensors of its own (float16 unless dtype says otherwise)."""
        import torch
        shape = (layers, pages, kv_heads, page, dim)
        k = torch.zeros(shape, dtype=dtype or torch.float16, device=device)
        meta = torch.zeros(cls.meta_words(slots, max_pages, pages), dtype=torch.int32, device=device)
        cache = cls(k, torch.zeros_like(k), meta, slots, max_pages)
        cache.free.copy_(torch.arange(pages - 1, -1, -1, dtype=torch.int32))
        cache.words[0] = pages
        return cache

    def extend(self, seqs, counts, stream=None):
        """Room for counts[i] more tokens in slot seqs[i]."""
        n = seqs.numel()
        dev = _gpu("extend: tensors of one GPU", self.meta, seqs, counts)
        _check(_on(dev, self._lib.pi_cache_extend, self._ref, _ints(seqs, n, "extend: seqs"),
                   _ints(counts, n, "extend: counts"), n, _stream_on(dev, stream)), "pi_cache_extend")

    def append(self, layer: int, k, v, cu, seqs, stream=None):
        """Rows cu[i] .. cu[i + 1] - 1 of k and v [tokens][kv_heads][dim] become the last tokens of slot seqs[i]."""
        shape = k.shape
        _need(len(shape) == 3 and shape == v.shape and shape[1] == self.kv_heads and shape[2] == self.dim
              and k.dtype == v.dtype == self.dtype, "append: k, v")
        n = seqs.numel()
        dev = _gpu("append: tensors of one GPU", self.meta, k, v, cu, seqs)
        _check(_on(dev, self._lib.pi_cache_append, self._ref, layer, _heads(k, shape, "append: k"),
                   _heads(v, shape, "append: v"), shape[0], _ints(cu, n + 1, "append: cu"), _ints(seqs, n, "append: seqs"), n,
                   _stream_on(dev, stream)), "pi_cache_append")

    def fork(self, parents, children, stream=None):
        """The empty slot children[i] becomes a copy of slot parents[i]."""
        n = parents.numel()
        dev = _gpu("fork: tensors of one GPU", self.meta, parents, children)
        on = _stream_on(dev, stream)
        _check(_on(dev, self._lib.pi_cache_fork, self._ref, _ints(parents, n, "fork: parents"),
                   _ints(children, n, "fork: children"), n, self._ws.on(on), self._ws.bytes, on), "pi_cache_fork")

    def release(self, seqs, stream=None):
        """The listed slots become empty."""
        n = seqs.numel()
        dev = _gpu("release: tensors of one GPU", self.meta, seqs)
        _check(_on(dev, self._lib.pi_cache_release, self._ref, _ints(seqs, n, "release: seqs"), n,
                   _stream_on(dev, stream)), "pi_cache_release")

    def compact(self, moved=None, stream=None):
        """The pages in use move to the front of the pool; moved [pages]: the new place of each."""
        dev = _gpu("compact: tensors of one GPU", self.meta, moved)
        on = _stream_on(dev, stream)
        _check(_on(dev, self._lib.pi_cache_compact, self._ref, _ints(moved, self.pages, "compact: moved"), self._ws.on(on),
                   self._ws.bytes, on), "pi_cache_compact")

    def errors(self) -> int:
        """The error word (waits for the device)."""
        return int(self.words[1])

    def reserve(self, batch: int, heads: int):
        """Memory for attn_decode of up to `batch` rows of `heads` heads, so that no call of these has to take any."""
        _need(batch > 0, "reserve: batch")
        n = max(self._attn_needs(b, heads) for b in range(1, batch + 1))
        if self._attn_ws is None or n > self._attn_ws.bytes:
            self._attn_grow(n, None)

    def attn_workspace(self, batch: int, heads: int):
        """The workspace of attn_decode for these sizes: a buffer of at least as many bytes, the same for all sizes."""
        return self._attn_scratch(batch, heads, None).mem

    def _attn_scratch(self, batch: int, heads: int, handle: Optional[int]) -> _Scratch:
        """That workspace, for a call on a stream (None: the current one)."""
        n = self._attn_need.get((batch, heads)) or self._attn_needs(batch, heads)
        if self._attn_ws is None or n > self._attn_ws.bytes:
            self._attn_grow(n, handle)
        return self._attn_ws

    def _attn_needs(self, batch: int, heads: int) -> int:
        n = int(lib().pi_attn_workspace_bytes(self._ref, batch, heads))
        _need(n > 0, "attn_decode: batch, heads")
        self._attn_need[batch, heads] = n
        return n

    def _attn_grow(self, n: int, handle: Optional[int]):
        # memory taken while a graph is captured belongs to that graph
        _need(not (_capturing(self._ws.dev) or handle is not None and _capturing(self._ws.dev, handle)),
              "attn_decode: a call inside a capture needs more workspace")
        # graphs hold the buffers before this one, so these stay; twice the size each time, they are smaller than it together
        if self._attn_ws is not None:
            self._attn_before.append(self._attn_ws)
            n = max(n, 2 * self._attn_ws.bytes)
        self._attn_ws = _Scratch(n, self.k_pool.device)


def attn_prompt(q, k, v, out, cu, scale: float = 0.0, stream=None):
    """Causal attention over packed sequences, rows cu[i] .. cu[i + 1] - 1 each.

    q, out: [tokens][heads][dim]; k, v: [tokens][kv_heads][dim]; scale 0: 1 / sqrt(dim)."""
    qs, ks, n = q.shape, k.shape, cu.numel() - 1
    _need(len(qs) == len(ks) == 3 and qs == out.shape and ks == v.shape and qs[0] == ks[0] and qs[2] == ks[2]
          and q.dtype == k.dtype == v.dtype == out.dtype, "attn_prompt: q, k, v, out")
    _need(n > 0, "attn_prompt: cu")
    offsets, what = _ints(cu, None, "attn_prompt: cu"), "attn_prompt: strides"
    dev = _gpu("attn_prompt: tensors of one GPU", cu, q, k, v, out)
    _check(_on(dev, (_lib or lib()).pi_attn_prompt, _heads(q, qs, what), _heads(k, ks, what), _heads(v, ks, what),
               _heads(out, qs, what), qs[0], qs[1], ks[1], qs[2], _dtype_of(q), offsets, n, scale,
               _stream_on(dev, stream)), "pi_attn_prompt")


def attn_decode(cache: Cache, layer: int, q, out, prefix=None, seqs=None, scale: float = 0.0, ws=None, stream=None):
    """Attention of one query row [heads][dim] per batch row over what its slot holds in a layer.

    seqs: the slots (None: row b is slot b).  prefix: an int32 tensor of one element, how many
    leading pages the slots that are not empty have in common (PI_CACHE_EPREFIX in the error
    word where they do not).  ws: as Cache.attn_workspace."""
    shape = q.shape
    _need(len(shape) == 3 and shape == out.shape and shape[2] == cache.dim and q.dtype == out.dtype == cache.dtype,
          "attn_decode: q, out")
    dev = _gpu("attn_decode: tensors of one GPU", cache.meta, q, out, prefix, seqs, ws)
    batch, heads, _ = shape
    on = _stream_on(dev, stream)
    if ws is None:
        scratch = cache._attn_scratch(batch, heads, on)
        memory, size = scratch.on(on), scratch.bytes
    else:
        _need(ws.is_contiguous(), "attn_decode: ws")   # any other's elements lie elsewhere than one after the other
        memory, size = ws.data_ptr(), ws.numel() * ws.element_size()
    what = "attn_decode: strides"
    _check(_on(dev, cache._lib.pi_attn_decode, cache._ref, layer, _heads(q, shape, what), _heads(out, shape, what), batch,
               heads, _ints(seqs, batch, "attn_decode: seqs"), _ints(prefix, 1, "attn_decode: prefix"), scale,
               memory, size, on), "pi_attn_decode")


class Q4Matrix:
    """A Q4_0 matrix [rows][cols] with the workspace of its products of up to `batch` rows.

    nibbles: uint8 [rows][cols / 2]; scales: float16 (or its bits) [rows][cols / 32]; bias: float32
    [rows] or None.  Products with one matrix belong on one stream."""

    def __init__(self, nibbles, scales, bias=None, batch: int = 1):
        import torch
        _need(nibbles.dtype == torch.uint8 and nibbles.dim() == 2 and nibbles.is_contiguous(), "Q4Matrix: nibbles")
        self.rows, self.cols, self.batch = nibbles.shape[0], 2 * nibbles.shape[1], int(batch)
        _need(scales.dtype in (torch.float16, torch.int16) and scales.is_contiguous()
              and tuple(scales.shape) == (self.rows, self.cols // 32), "Q4Matrix: scales")
        _need(bias is None or (bias.dtype == torch.float32 and bias.is_contiguous()
                               and tuple(bias.shape) == (self.rows,)), "Q4Matrix: bias")
        n = int(lib().pi_matvec_workspace_bytes(self.rows, self.cols, self.batch))
        _need(n > 0, "Q4Matrix: rows, cols, batch")
        _gpu("Q4Matrix: tensors of one GPU", nibbles, scales, bias)
        self.nibbles, self.scales, self.bias = nibbles, scales, bias
        self.struct = PiMat(_p(nibbles), _p(scales))
        self._ws = _Scratch(n, nibbles.device)
        self.ws = self._ws.mem
        self._args = ctypes.byref(self.struct), self.rows, self.cols, _p(bias)
        self._lib = lib()

    @classmethod
    def upload(cls, mat, bias=None, batch: int = 1, device="cuda") -> "Q4Matrix":
        """Copy a host Q4_0 matrix (.nibbles, .scales as NumPy arrays) to the GPU."""
        import numpy as np
        import torch
        nib = torch.from_numpy(np.ascontiguousarray(mat.nibbles)).to(device)
        sc = torch.from_numpy(np.ascontiguousarray(mat.scales).view(np.int16)).to(device)
        return cls(nib, sc, None if bias is None else torch.from_numpy(np.ascontiguousarray(bias)).to(device), batch)


def matvec(mat: Q4Matrix, x, y, stream=None):
    """y[b] = W x[b] + bias; x [batch][cols], y [batch][rows], float32, float16 or bfloat16 each."""
    xs, ys = x.shape, y.shape
    _need(len(xs) == len(ys) == 2 and xs[0] == ys[0] <= mat.batch and xs[1] == mat.cols and ys[1] == mat.rows,
          "matvec: x, y")
    (ldx, x1), (ldy, y1), batch = x.stride(), y.stride(), xs[0]
    _need(x1 == 1 and (y1 == 1 or ys[1] == 1), "matvec: strides")
    if batch == 1:                                     # a row's stride says nothing there
        ldx, ldy = xs[1], ys[1]
    dev = _gpu("matvec: tensors of one GPU", mat.nibbles, x, y)
    on = _stream_on(dev, stream)
    _check(_on(dev, mat._lib.pi_matvec, *mat._args, x.data_ptr(), _dtype_of(x), ldx, y.data_ptr(), _dtype_of(y), ldy,
               batch, mat._ws.on(on), mat._ws.bytes, on), "pi_matvec")


# ------------------------------------------------------- HIP runtime plumbing
_hip = None


def hip_runtime():
    """The HIP runtime (libamdhip64) for graphs and timing events."""
    global _hip
    if _hip is None:
        H = ctypes.CDLL("libamdhip64.so")
        P = ctypes.c_void_p
        H.hipGetErrorString.restype = ctypes.c_char_p
        H.hipEventCreate.argtypes = [ctypes.POINTER(P)]
        H.hipEventDestroy.argtypes = [P]
        H.hipEventRecord.argtypes = [P, P]
        H.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), P, P]
        H.hipStreamBeginCapture.argtypes = [P, ctypes.c_int]
        H.hipStreamEndCapture.argtypes = [P, ctypes.POINTER(P)]
        H.hipGraphInstantiate.argtypes = [ctypes.POINTER(P), P, P, P, ctypes.c_size_t]
        H.hipGraphLaunch.argtypes = [P, P]
        H.hipGraphExecDestroy.argtypes = [P]
        H.hipGraphDestroy.argtypes = [P]
        H.hipStreamCreate.argtypes = [ctypes.POINTER(P)]
        H.hipStreamDestroy.argtypes = [P]
        H.hipStreamSynchronize.argtypes = [P]
        _hip = H
    return _hip


def _hip_check(r: int, where: str):
    if r != 0:
        raise RuntimeError(f"{where}: {hip_runtime().hipGetErrorString(r).decode()} ({r})")


class HipEvent:
    """A timing hipEvent_t; int(ev) is the handle."""

    def __init__(self):
        self.h = ctypes.c_void_p()
        _hip_check(hip_runtime().hipEventCreate(ctypes.byref(self.h)), "hipEventCreate")

    def __int__(self):
        return int(self.h.value)

    def record(self, stream):
        _hip_check(hip_runtime().hipEventRecord(self.h, _stream(stream)), "hipEventRecord")

    def elapsed_ms(self, later: "HipEvent") -> float:
        ms = ctypes.c_float()
        _hip_check(hip_runtime().hipEventElapsedTime(ctypes.byref(ms), self.h, later.h), "hipEventElapsedTime")
        return float(ms.value)

    def __del__(self):
        if _hip is not None and self.h:
            _hip.hipEventDestroy(self.h)


class HipStream:
    """A plain hipStream_t (default flags and priority); .cuda_stream is the handle."""

    def __init__(self):
        self.h = ctypes.c_void_p()
        _hip_check(hip_runtime().hipStreamCreate(ctypes.byref(self.h)), "hipStreamCreate")

    @property
    def cuda_stream(self) -> int:
        return int(self.h.value)

    def synchronize(self):
        _hip_check(hip_runtime().hipStreamSynchronize(self.h), "hipStreamSynchronize")

    def __del__(self):
        if _hip is not None and self.h:
            _hip.hipStreamDestroy(self.h)


class HipGraph:
    """Stream capture of fn(stream) into an instantiated hipGraph, replayed on that stream.

    Only library calls belong inside fn: nothing in it may allocate."""

    def __init__(self, stream, fn):
        H = hip_runtime()
        self.stream = _stream(stream)
        self.g, self.ge = ctypes.c_void_p(), ctypes.c_void_p()
        _hip_check(H.hipStreamBeginCapture(self.stream, 0), "hipStreamBeginCapture")  # global mode
        try:
            fn(stream)
        finally:
            _hip_check(H.hipStreamEndCapture(self.stream, ctypes.byref(self.g)), "hipStreamEndCapture")
        _hip_check(H.hipGraphInstantiate(ctypes.byref(self.ge), self.g, None, None, 0), "hipGraphInstantiate")

    def replay(self):
        _hip_check(hip_runtime().hipGraphLaunch(self.ge, self.stream), "hipGraphLaunch")

    def __del__(self):
        if _hip is not None:
            if self.ge:
                _hip.hipGraphExecDestroy(self.ge)
            if self.g:
                _hip.hipGraphDestroy(self.g)


EXPORTED = ("pi_workspace_bytes", "pi_predict", "pi_sparse_ffn", "pi_ffn_stack", "pi_ffn_stack_static",
            "pi_cache_meta_words", "pi_cache_workspace_bytes", "pi_cache_extend", "pi_cache_append", "pi_cache_fork",
            "pi_cache_release", "pi_cache_compact", "pi_attn_prompt", "pi_attn_workspace_bytes", "pi_attn_decode",
            "pi_matvec_workspace_bytes", "pi_matvec", "pi_status_str", "pi_abi_version", "pi_last_hip_error")
