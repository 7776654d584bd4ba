"""Binding of ``liblrkv_serve.so`` (declared in ``include/lrkv_serve.h``): prefill
attention with score modifiers, the paged 8-bit cache and its page operations.

Like the rest of the package it only marshals arguments and checks their shapes
and types; the same names as in the C ABI are re-exported by the package.
"""
import ctypes
import functools
import os
import warnings
from dataclasses import dataclass, fields

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
SERVE_LIB_PATH = os.path.join(_PKG, "liblrkv_serve.so")

DEV_BAD_PAGE = 0x10
DEV_NO_PAGES = 0x20
DEV_BAD_SEQ = 0x40
CODES = {"int8": 0, "e4m3": 1}

_P, _I, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t


class _Score(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", _I), ("slopes", _P),
                ("first_key", _P), ("prefix_end", _P)]


class _PrefillDims(ctypes.Structure):
    # the strides one by one (q_stride[0] is q_stride0): making four arrays a call takes 2 us
    _fields_ = [(n, _I) for n in ("B", "Hq", "Hkv", "d", "t_q", "t_k")] + \
        [(f"{n}_stride{i}", ctypes.c_int64) for n in ("q", "k", "v", "out") for i in range(3)]


class _PagedDims(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("B", "Hq", "Hkv", "d", "page", "n_pages", "max_pages", "n_layers", "code")]


class _PagedCache(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k", "v", "scale_k", "scale_v", "page_table", "seq_len", "refs", "dev_status")]


_lib = None
_calls = None    # the calls marshalled in C++ (csrc/serve/serve_calls.cpp)

_SIGNATURES = {
    "lrkv_prefill_workspace_size": (_SZ, [_P]),
    "lrkv_prefill_attn": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "lrkv_paged_append": (_I, [_P, _P, _I, _P, _P, _I, _P, _P]),
    "lrkv_paged_read": (_I, [_P, _P, _I, _P, _P, _I, _P, _P, _P]),
    "lrkv_paged_workspace_size": (_SZ, [_P, _I]),
    "lrkv_paged_attn": (_I, [_P, _P, _I, _P, _I, _P, _P, _P, _P, _SZ, _P]),
    "lrkv_pages_reserve": (_I, [_P, _P, _I, _P, _P]),
    "lrkv_pages_advance": (_I, [_P, _P, _I, _P, _P]),
    "lrkv_pages_fork": (_I, [_P, _P, _P, _P, _I, _P, _SZ, _P]),
    "lrkv_pages_free": (_I, [_P, _P, _P, _I, _P]),
    "lrkv_pages_copy": (_I, [_P, _P, _P, _P, _I, _P, _SZ, _P]),
    "lrkv_pages_compact": (_I, [_P, _P, _P, _SZ, _P]),
}


class _InPython:
    """In place of the calls in C++: every one is for the Python path."""

    def __getattr__(self, name):
        return lambda *args: -1


def load_serve_library(path=None):
    """Load liblrkv_serve.so (built in-tree).  Raises if it has not been built."""
    global _lib, _calls
    if _lib is not None and path is None:
        return _lib
    p = path or SERVE_LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with `python -m decode_attention_lrkv_b200.build`")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    if path is None:
        try:
            from . import _serve_calls
            _serve_calls.bind([ctypes.cast(getattr(lib, "lrkv_" + n), _P).value for n in (
                "prefill_workspace_size", "prefill_attn", "paged_append", "paged_read", "paged_attn", "pages_reserve",
                "pages_advance", "pages_fork", "pages_copy", "pages_free", "pages_compact")])
        except (ImportError, ValueError) as e:   # missing, or built for another torch
            warnings.warn(f"_serve_calls.so cannot be used ({e}): the calls are marshalled in Python, which takes "
                          "several microseconds more of host time; build it with "
                          "`python -m decode_attention_lrkv_b200.build`", RuntimeWarning, stacklevel=2)
            _serve_calls = _InPython()
        _lib, _calls = lib, _serve_calls
    return lib


def _fast():
    """The calls in C++.  They return -1 for arguments that the Python path has to look at."""
    if _calls is None:
        load_serve_library()
    return _calls


class _Fields:
    """Copies and pickles take a dataclass's fields; what __post_init__ derives from them is made anew."""

    def __getstate__(self):
        return {f.name: getattr(self, f.name) for f in fields(self)}

    def __setstate__(self, state):
        for name, value in state.items():
            object.__setattr__(self, name, value)
        self.__post_init__()


@dataclass(frozen=True)
class Score(_Fields):
    """Score modifiers (``lrkv_score``): scale 0 stands for 1/sqrt(d), softcap and
    window 0 for none; slopes [Hq] fp32; first_key and prefix_end [B, t_q] int32."""
    scale: float = 0.0
    softcap: float = 0.0
    window: int = 0
    slopes: torch.Tensor = None
    first_key: torch.Tensor = None
    prefix_end: torch.Tensor = None

    def __post_init__(self):
        _int32(self.window, "window")
        plain = self.slopes is None and self.first_key is None and self.prefix_end is None
        object.__setattr__(self, "_struct", self.c() if plain else None)
        object.__setattr__(self, "_plain", ctypes.byref(self._struct) if plain else None)
        object.__setattr__(self, "_score_at", ctypes.addressof(self._struct) if plain else None)

    def c(self):
        return _Score(self.scale, self.softcap, self.window, _addr(self.slopes), _addr(self.first_key),
                      _addr(self.prefix_end))


@dataclass(frozen=True)
class PagedDims(_Fields):
    B: int
    Hq: int
    Hkv: int
    d: int
    page: int
    n_pages: int
    max_pages: int
    n_layers: int = 1
    code: str = "int8"

    def __post_init__(self):
        object.__setattr__(self, "_struct", self.c())
        object.__setattr__(self, "_ref", ctypes.byref(self._struct))
        object.__setattr__(self, "_at", ctypes.addressof(self._struct))

    def c(self):
        sizes = ("B", "Hq", "Hkv", "d", "page", "n_pages", "max_pages", "n_layers")
        return _PagedDims(*(_int32(getattr(self, n), n) for n in sizes), CODES[self.code])


class PagedCache:
    """The pool, page table and counts of ``lrkv_paged_cache`` as torch tensors.

    k, v: uint8 [n_layers, n_pages, Hkv, page, d]; scale_k, scale_v: fp32 [n_layers,
    n_pages, Hkv]; int32 page_table [B, max_pages] (-1: no page), seq_len [B], refs
    [n_pages]; dev_status int32 [4] (word 0 used).  Tensors that the caller already
    has may be given by name; the others are made for a new, empty cache.  All lie on one
    device.  A tensor may be replaced by one of the same shape, type and device; dims stay.
    """
    FIELDS = ("k", "v", "scale_k", "scale_v", "page_table", "seq_len", "refs", "dev_status")

    def __init__(self, dims, device="cuda", **given):
        D = dims
        shapes = {"k": ((D.n_layers, D.n_pages, D.Hkv, D.page, D.d), torch.uint8),
                  "scale_k": ((D.n_layers, D.n_pages, D.Hkv), torch.float32),
                  "page_table": ((D.B, D.max_pages), torch.int32), "seq_len": ((D.B,), torch.int32),
                  "refs": ((D.n_pages,), torch.int32), "dev_status": ((4,), torch.int32)}
        shapes["v"], shapes["scale_v"] = shapes["k"], shapes["scale_k"]
        unknown = [name for name in given if name not in shapes]
        if unknown:
            raise TypeError(f"PagedCache has no {', '.join(unknown)}")
        given = {name: t for name, t in given.items() if t is not None}
        if given:
            device = next(iter(given.values())).device
        self._shapes, self.dims = shapes, dims
        for name in self.FIELDS:
            shape, dtype = shapes[name]
            t = given.get(name)
            if t is None:
                t = torch.full(shape, -1 if name == "page_table" else 0, dtype=dtype, device=device)
            setattr(self, name, t)

    def __setattr__(self, name, value):
        # the calls take the tensors' addresses, and the sizes from dims
        if name in self.FIELDS:
            _check(value, name, *self._shapes[name])
            device = self.__dict__.setdefault("_device", value.device)   # that of the first one
            if value.device != device:
                raise ValueError(f"{name}: the cache's other tensors are on {device}, this one is on {value.device}")
        elif name in ("dims", "_shapes") and name in self.__dict__:
            raise AttributeError(f"a PagedCache's {name} cannot be replaced")
        object.__setattr__(self, name, value)

    def c(self):
        return _PagedCache(self.k.data_ptr(), self.v.data_ptr(), self.scale_k.data_ptr(), self.scale_v.data_ptr(),
                           self.page_table.data_ptr(), self.seq_len.data_ptr(), self.refs.data_ptr(),
                           self.dev_status.data_ptr())

    def nbytes(self):
        return sum(getattr(self, f).numel() * getattr(self, f).element_size() for f in self.FIELDS)


def _int32(value, name):
    """ctypes cuts a whole number to 32 bits without a word."""
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{name}: {value} does not fit in 32 bits")
    return value


def _addr(t):
    return None if t is None else t.data_ptr()


def _check(t, name, shape, dtype, device=None):
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} is needed, got "
                         f"{t.dtype} {tuple(t.shape)}" + ("" if t.is_contiguous() else ", not contiguous"))
    if device is not None and t.get_device() != device:
        _wrong_device(t, name, device)


def _wrong_device(t, name, device):
    raise ValueError(f"{name}: a CUDA tensor on cuda:{device} is needed, got one on {t.device}")


def _device(t, name):
    """The device that the call's tensors have to be on: the library launches on the current one."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name}: a CUDA tensor is needed, got one on {t.device}")
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return device


def _check_score(score, B, t_q, Hq, device):
    if score is None:
        return
    if not isinstance(score, Score):
        raise TypeError(f"score: a Score is needed, got {type(score).__name__}")
    if score._plain is not None:
        return
    if score.slopes is not None:
        _check(score.slopes, "slopes", (Hq,), torch.float32, device)
    if score.first_key is not None:
        _check(score.first_key, "first_key", (B, t_q), torch.int32, device)
    if score.prefix_end is not None:
        _check(score.prefix_end, "prefix_end", (B, t_q), torch.int32, device)


def _check_list(t, name, n, device):
    if t is not None:
        _check(t, name, (n,), torch.int32, device)


def _check_status(t, device):
    if t is None:
        return
    if t.dtype != torch.int32 or not t.is_contiguous() or t.numel() < 1:
        raise ValueError(f"dev_status: a contiguous int32 tensor of a word at least is needed, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != device:
        _wrong_device(t, "dev_status", device)


def _check_ws(ws, device):
    if ws is None:
        return 0
    if ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("ws: a contiguous uint8 tensor is needed")
    if ws.get_device() != device:
        _wrong_device(ws, "ws", device)
    return ws.numel()


def _stream(stream, device):
    # current_stream() builds an object (3 us); the raw handle is what the library takes
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise ValueError(f"stream is one of cuda:{stream.device_index}, the tensors are on cuda:{device}")
    return stream.cuda_stream


def _ref(score):
    if score is None:
        return None
    return score._plain if score._plain is not None else ctypes.byref(score.c())


def _cache_ref(dims, cache, device):
    if cache.dims is not dims and cache.dims != dims:
        raise ValueError(f"the cache was made for {cache.dims}, not {dims}")
    for name in cache.FIELDS:
        t = getattr(cache, name)
        if t.get_device() != device:
            _wrong_device(t, name, device)
    return ctypes.byref(cache.c())


def _done(code, what, check):
    if check and code != 0:
        from . import LrkvError
        raise LrkvError(code, what)
    return code


def _prefill_dims(q, k, v, out):
    B, t_q, Hq, d = q.shape
    _, t_k, Hkv, _ = k.shape
    for x in (B, t_q, Hq, t_k, Hkv, d):
        _int32(x, "a size of q or k")
    return _PrefillDims(B, Hq, Hkv, d, t_q, t_k, *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *out.stride()[:3])


@functools.lru_cache(maxsize=1024)
def _prefill_ws(device, B, Hq, t_q, t_k):
    """Bytes of workspace, which go by the sizes and the current device's SMs alone."""
    dense = _PrefillDims(B, Hq, Hq, 128, t_q, t_k, *(4 * (max(t_q, t_k, 1) * Hq * 128, Hq * 128, 128)))
    return load_serve_library().lrkv_prefill_workspace_size(ctypes.byref(dense))


def _check_rows(t, name, device):
    if t.dtype != torch.bfloat16 or t.dim() != 4 or (t.stride(3) != 1 and t.shape[3] > 1):
        raise ValueError(f"{name}: a bf16 tensor [B, t, heads, d] with contiguous rows is needed")
    if t.get_device() != device:
        _wrong_device(t, name, device)


def lrkv_prefill_workspace_size(q, k, v, out):
    return int(load_serve_library().lrkv_prefill_workspace_size(ctypes.byref(_prefill_dims(q, k, v, out))))


def lrkv_prefill_attn(q, k, v, out, q_len=None, kv_len=None, score=None, dev_status=None, ws=None, stream=None,
                      check=True):
    """out [B,t_q,Hq,d] <- attention of q [B,t_q,Hq,d] over k, v [B,t_k,Hkv,d] (bf16, rows of d contiguous
    elements, otherwise any strides); see include/lrkv_serve.h.  A workspace is made when one is needed
    and none is given."""
    code = _fast().prefill(q, k, v, out, q_len, kv_len, score, dev_status, ws, stream)
    if code >= 0:
        return _done(code, "lrkv_prefill_attn", check)
    device = _device(q, "q")
    _check_rows(q, "q", device)
    _check_rows(k, "k", device)
    _check_rows(v, "v", device)
    _check_rows(out, "out", device)
    B, t_q, Hq, d = q.shape
    if out.shape != q.shape or k.shape != v.shape or k.shape[0] != B or k.shape[3] != d:
        raise ValueError(f"shapes do not fit: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}, "
                         f"out {tuple(out.shape)}")
    _check_list(q_len, "q_len", B, device)
    _check_list(kv_len, "kv_len", B, device)
    _check_score(score, B, t_q, Hq, device)
    _check_status(dev_status, device)
    n_ws = _check_ws(ws, device)
    lib, dims = load_serve_library(), ctypes.byref(_prefill_dims(q, k, v, out))
    if ws is None:
        n_ws = _prefill_ws(device, B, Hq, t_q, k.shape[1])
        if n_ws:   # memory of the stream that uses it: it may be handed on as soon as this call returns
            with torch.cuda.stream(stream):
                ws = torch.empty(n_ws, dtype=torch.uint8, device=q.device)
    return _done(lib.lrkv_prefill_attn(dims, q.data_ptr(), k.data_ptr(), v.data_ptr(), _addr(q_len), _addr(kv_len),
                                       _ref(score), out.data_ptr(), _addr(dev_status), _addr(ws), n_ws,
                                       _stream(stream, device)), "lrkv_prefill_attn", check)


def lrkv_paged_workspace_size(dims, t_q=1):
    return int(load_serve_library().lrkv_paged_workspace_size(dims._ref, _int32(int(t_q), "t_q")))


def make_paged_workspace(dims, t_q=1, device="cuda"):
    """A zero-filled workspace for the paged calls on `dims` with up to t_q query rows a sequence."""
    n = lrkv_paged_workspace_size(dims, t_q)
    if n == 0:
        raise ValueError(f"invalid dims {dims}, t_q {t_q}")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def lrkv_paged_append(dims, cache, layer, k_new, v_new, t_new_b=None, stream=None, check=True):
    """Quantise k_new, v_new [B,t_new,Hkv,d] (bf16) into `layer`'s pages at positions seq_len .. ."""
    code = _fast().append(dims, cache, layer, k_new, v_new, t_new_b, stream)
    if code >= 0:
        return _done(code, "lrkv_paged_append", check)
    t_new = k_new.shape[1]
    shape = (dims.B, t_new, dims.Hkv, dims.d)
    device = _device(cache.k, "cache")
    _check(k_new, "k_new", shape, torch.bfloat16, device)
    _check(v_new, "v_new", shape, torch.bfloat16, device)
    _check_list(t_new_b, "t_new_b", dims.B, device)
    return _done(load_serve_library().lrkv_paged_append(
        dims._ref, _cache_ref(dims, cache, device), _int32(layer, "layer"), k_new.data_ptr(), v_new.data_ptr(), t_new,
        _addr(t_new_b), _stream(stream, device)), "lrkv_paged_append", check)


def lrkv_paged_read(dims, cache, layer, first, count, k_out, v_out, stream=None, check=True):
    """Positions first[b] .. first[b] + count[b] - 1 of `layer` as bf16 rows of k_out, v_out [B,t,Hkv,d]."""
    code = _fast().read(dims, cache, layer, first, count, k_out, v_out, stream)
    if code >= 0:
        return _done(code, "lrkv_paged_read", check)
    t_max = k_out.shape[1]
    shape = (dims.B, t_max, dims.Hkv, dims.d)
    device = _device(cache.k, "cache")
    _check(k_out, "k_out", shape, torch.bfloat16, device)
    _check(v_out, "v_out", shape, torch.bfloat16, device)
    _check_list(first, "first", dims.B, device)
    _check_list(count, "count", dims.B, device)
    return _done(load_serve_library().lrkv_paged_read(
        dims._ref, _cache_ref(dims, cache, device), _int32(layer, "layer"), _addr(first), _addr(count), t_max,
        k_out.data_ptr(), v_out.data_ptr(), _stream(stream, device)), "lrkv_paged_read", check)


def lrkv_paged_attn(dims, cache, layer, q, out, t_q_b=None, score=None, ws=None, stream=None, check=True):
    """out [B,t_q,Hq,d] <- attention of the newest t_q tokens' queries q (bf16) over `layer`'s pages."""
    code = _fast().attn(dims, cache, layer, q, out, t_q_b, score, ws, stream)
    if code >= 0:
        return _done(code, "lrkv_paged_attn", check)
    t_q = q.shape[1]
    shape = (dims.B, t_q, dims.Hq, dims.d)
    device = _device(cache.k, "cache")
    _check(q, "q", shape, torch.bfloat16, device)
    _check(out, "out", shape, torch.bfloat16, device)
    _check_list(t_q_b, "t_q_b", dims.B, device)
    _check_score(score, dims.B, t_q, dims.Hq, device)
    n_ws = _check_ws(ws, device)
    return _done(load_serve_library().lrkv_paged_attn(
        dims._ref, _cache_ref(dims, cache, device), _int32(layer, "layer"), q.data_ptr(), t_q, _addr(t_q_b),
        _ref(score), out.data_ptr(), _addr(ws), n_ws, _stream(stream, device)), "lrkv_paged_attn", check)


def _count_call(fn, name, dims, cache, t_new, t_new_b, stream, check):
    device = _device(cache.k, "cache")
    _check_list(t_new_b, "t_new_b", dims.B, device)
    return _done(fn(dims._ref, _cache_ref(dims, cache, device), _int32(t_new, "t_new"), _addr(t_new_b),
                    _stream(stream, device)), name, check)


def lrkv_pages_reserve(dims, cache, t_new, t_new_b=None, stream=None, check=True):
    """Pages for t_new (or t_new_b[b]) more tokens of every sequence."""
    code = _fast().counts(0, dims, cache, t_new, t_new_b, stream)
    if code >= 0:
        return _done(code, "lrkv_pages_reserve", check)
    return _count_call(load_serve_library().lrkv_pages_reserve, "lrkv_pages_reserve", dims, cache, t_new, t_new_b,
                       stream, check)


def lrkv_pages_advance(dims, cache, t_new, t_new_b=None, stream=None, check=True):
    """seq_len += t_new (or t_new_b), up to the first token that has no page."""
    code = _fast().counts(1, dims, cache, t_new, t_new_b, stream)
    if code >= 0:
        return _done(code, "lrkv_pages_advance", check)
    return _count_call(load_serve_library().lrkv_pages_advance, "lrkv_pages_advance", dims, cache, t_new, t_new_b,
                       stream, check)


def _pair_call(fn, name, dims, cache, src, dst, ws, stream, check):
    device, n = _device(cache.k, "cache"), src.numel()
    _check_list(src, "src", n, device)
    _check_list(dst, "dst", n, device)
    n_ws = _check_ws(ws, device)
    return _done(fn(dims._ref, _cache_ref(dims, cache, device), src.data_ptr(), dst.data_ptr(), _int32(n, "src"),
                    _addr(ws), n_ws, _stream(stream, device)), name, check)


def lrkv_pages_fork(dims, cache, src, dst, ws=None, stream=None, check=True):
    """Sequence dst[i] becomes a copy of sequence src[i] (int32 lists on the device)."""
    code = _fast().lists(0, dims, cache, src, dst, ws, stream)
    if code >= 0:
        return _done(code, "lrkv_pages_fork", check)
    return _pair_call(load_serve_library().lrkv_pages_fork, "lrkv_pages_fork", dims, cache, src, dst, ws, stream, check)


def lrkv_pages_copy(dims, cache, src, dst, ws=None, stream=None, check=True):
    """Copy pages src[i] to dst[i] (int32 lists on the device) in every layer."""
    code = _fast().lists(1, dims, cache, src, dst, ws, stream)
    if code >= 0:
        return _done(code, "lrkv_pages_copy", check)
    return _pair_call(load_serve_library().lrkv_pages_copy, "lrkv_pages_copy", dims, cache, src, dst, ws, stream, check)


def lrkv_pages_free(dims, cache, seqs, stream=None, check=True):
    """Empty the sequences listed in seqs (int32, on the device)."""
    code = _fast().lists(2, dims, cache, seqs, None, None, stream)
    if code >= 0:
        return _done(code, "lrkv_pages_free", check)
    device, n = _device(cache.k, "cache"), seqs.numel()
    _check_list(seqs, "seqs", n, device)
    return _done(load_serve_library().lrkv_pages_free(
        dims._ref, _cache_ref(dims, cache, device), seqs.data_ptr(), _int32(n, "seqs"), _stream(stream, device)),
        "lrkv_pages_free", check)


def lrkv_pages_compact(dims, cache, ws=None, stream=None, check=True):
    """Move pages so that the live ones have the lowest ids."""
    code = _fast().lists(3, dims, cache, None, None, ws, stream)
    if code >= 0:
        return _done(code, "lrkv_pages_compact", check)
    device = _device(cache.k, "cache")
    n_ws = _check_ws(ws, device)
    return _done(load_serve_library().lrkv_pages_compact(dims._ref, _cache_ref(dims, cache, device), _addr(ws), n_ws,
                                                         _stream(stream, device)), "lrkv_pages_compact", check)
