"""Binding of ``liblrkv_serve.so`` (declared in ``include/lrkv_serve.h``): prefill
attention with score modifiers, the paged 8-bit cache and its page operations.

Like the rest of the package it only marshals arguments and checks their shapes
and types; the same names as in the C ABI are re-exported by the package.
"""
import ctypes
import os
from dataclasses import dataclass

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
    _fields_ = [(n, _I) for n in ("B", "Hq", "Hkv", "d", "t_q", "t_k")] + \
        [(n, ctypes.c_int64 * 3) for n in ("q_stride", "k_stride", "v_stride", "out_stride")]


class _PagedDims(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("B", "Hq", "Hkv", "d", "page", "n_pages", "max_pages", "n_layers", "code")]


class _PagedCache(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k", "v", "scale_k", "scale_v", "page_table", "seq_len", "refs", "dev_status")]


_lib = None

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


def load_serve_library(path=None):
    """Load liblrkv_serve.so (built in-tree).  Raises if it has not been built."""
    global _lib
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
        _lib = lib
    return lib


@dataclass(frozen=True)
class Score:
    """Score modifiers (``lrkv_score``): scale 0 stands for 1/sqrt(d), softcap and
    window 0 for none; slopes [Hq] fp32; first_key and prefix_end [B, t_q] int32."""
    scale: float = 0.0
    softcap: float = 0.0
    window: int = 0
    slopes: torch.Tensor = None
    first_key: torch.Tensor = None
    prefix_end: torch.Tensor = None

    def c(self):
        return _Score(self.scale, self.softcap, self.window, _addr(self.slopes), _addr(self.first_key),
                      _addr(self.prefix_end))


@dataclass(frozen=True)
class PagedDims:
    B: int
    Hq: int
    Hkv: int
    d: int
    page: int
    n_pages: int
    max_pages: int
    n_layers: int = 1
    code: str = "int8"

    def c(self):
        return _PagedDims(self.B, self.Hq, self.Hkv, self.d, self.page, self.n_pages, self.max_pages, self.n_layers,
                          CODES[self.code])


class PagedCache:
    """The pool, page table and counts of ``lrkv_paged_cache`` as torch tensors.

    k, v: uint8 [n_layers, n_pages, Hkv, page, d]; scale_k, scale_v: fp32 [n_layers,
    n_pages, Hkv]; int32 page_table [B, max_pages] (-1: no page), seq_len [B], refs
    [n_pages]; dev_status int32 [4] (word 0 used).  Tensors that the caller already
    has may be given by name; the others are made for a new, empty cache.
    """
    FIELDS = ("k", "v", "scale_k", "scale_v", "page_table", "seq_len", "refs", "dev_status")

    def __init__(self, dims, device="cuda", **given):
        D = dims
        shapes = {"k": ((D.n_layers, D.n_pages, D.Hkv, D.page, D.d), torch.uint8),
                  "scale_k": ((D.n_layers, D.n_pages, D.Hkv), torch.float32),
                  "page_table": ((D.B, D.max_pages), torch.int32), "seq_len": ((D.B,), torch.int32),
                  "refs": ((D.n_pages,), torch.int32), "dev_status": ((4,), torch.int32)}
        shapes["v"], shapes["scale_v"] = shapes["k"], shapes["scale_k"]
        if given:
            device = next(iter(given.values())).device
        for name in self.FIELDS:
            shape, dtype = shapes[name]
            t = given.pop(name, None)
            if t is None:
                t = torch.full(shape, -1 if name == "page_table" else 0, dtype=dtype, device=device)
            _check(t, name, shape, dtype)
            setattr(self, name, t)
        if given:
            raise TypeError(f"PagedCache has no {', '.join(given)}")
        self.dims = dims

    def c(self):
        return _PagedCache(*[getattr(self, f).data_ptr() for f in self.FIELDS])

    def nbytes(self):
        return sum(getattr(self, f).numel() * getattr(self, f).element_size() for f in self.FIELDS)


def _addr(t):
    return None if t is None else t.data_ptr()


def _check(t, name, shape, dtype):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} is needed, got "
                         f"{t.dtype} {tuple(t.shape)}" + ("" if t.is_contiguous() else ", not contiguous"))


def _check_score(score, B, t_q, Hq):
    if score is None:
        return
    for name, shape, dtype in (("slopes", (Hq,), torch.float32), ("first_key", (B, t_q), torch.int32),
                               ("prefix_end", (B, t_q), torch.int32)):
        t = getattr(score, name)
        if t is not None:
            _check(t, name, shape, dtype)


def _check_list(t, name, n):
    if t is not None:
        _check(t, name, (n,), torch.int32)


def _stream(stream):
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _ref(score):
    return None if score is None else ctypes.byref(score.c())


def _done(code, what, check):
    if check and code != 0:
        from . import LrkvError
        raise LrkvError(code, what)
    return code


def _strides(t):
    return (ctypes.c_int64 * 3)(*t.stride()[:3])


def _prefill_dims(q, k, v, out):
    B, t_q, Hq, d = q.shape
    return _PrefillDims(B, Hq, k.shape[2], d, t_q, k.shape[1], _strides(q), _strides(k), _strides(v), _strides(out))


def lrkv_prefill_workspace_size(q, k, v, out):
    return int(load_serve_library().lrkv_prefill_workspace_size(ctypes.byref(_prefill_dims(q, k, v, out))))


def lrkv_prefill_attn(q, k, v, out, q_len=None, kv_len=None, score=None, dev_status=None, ws=None, stream=None,
                      check=True):
    """out [B,t_q,Hq,d] <- attention of q [B,t_q,Hq,d] over k, v [B,t_k,Hkv,d] (bf16, rows of d contiguous
    elements, otherwise any strides); see include/lrkv_serve.h.  A workspace is made when one is needed
    and none is given."""
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t.dtype != torch.bfloat16 or t.dim() != 4 or (t.shape[3] > 1 and t.stride(3) != 1):
            raise ValueError(f"{name}: a bf16 tensor [B, t, heads, d] with contiguous rows is needed")
    B, t_q, Hq, d = q.shape
    if tuple(out.shape) != tuple(q.shape) or tuple(k.shape) != tuple(v.shape) or k.shape[0] != B or k.shape[3] != d:
        raise ValueError(f"shapes do not fit: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}, "
                         f"out {tuple(out.shape)}")
    _check_list(q_len, "q_len", B)
    _check_list(kv_len, "kv_len", B)
    _check_score(score, B, t_q, Hq)
    lib, dims = load_serve_library(), _prefill_dims(q, k, v, out)
    need = lib.lrkv_prefill_workspace_size(ctypes.byref(dims))
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    return _done(lib.lrkv_prefill_attn(ctypes.byref(dims), q.data_ptr(), k.data_ptr(), v.data_ptr(), _addr(q_len),
                                       _addr(kv_len), _ref(score), out.data_ptr(), _addr(dev_status), _addr(ws),
                                       0 if ws is None else ws.numel(), _stream(stream)), "lrkv_prefill_attn", check)


def lrkv_paged_workspace_size(dims, t_q=1):
    return int(load_serve_library().lrkv_paged_workspace_size(ctypes.byref(dims.c()), int(t_q)))


def make_paged_workspace(dims, t_q=1, device="cuda"):
    """A zero-filled workspace for the paged calls on `dims` with up to t_q query rows a sequence."""
    n = lrkv_paged_workspace_size(dims, t_q)
    if n == 0:
        raise ValueError(f"invalid dims {dims}, t_q {t_q}")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def lrkv_paged_append(dims, cache, layer, k_new, v_new, t_new_b=None, stream=None, check=True):
    """Quantise k_new, v_new [B,t_new,Hkv,d] (bf16) into `layer`'s pages at positions seq_len .. ."""
    t_new = k_new.shape[1]
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _check(t, name, (dims.B, t_new, dims.Hkv, dims.d), torch.bfloat16)
    _check_list(t_new_b, "t_new_b", dims.B)
    return _done(load_serve_library().lrkv_paged_append(
        ctypes.byref(dims.c()), ctypes.byref(cache.c()), layer, k_new.data_ptr(), v_new.data_ptr(), t_new,
        _addr(t_new_b), _stream(stream)), "lrkv_paged_append", check)


def lrkv_paged_read(dims, cache, layer, first, count, k_out, v_out, stream=None, check=True):
    """Positions first[b] .. first[b] + count[b] - 1 of `layer` as bf16 rows of k_out, v_out [B,t,Hkv,d]."""
    t_max = k_out.shape[1]
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        _check(t, name, (dims.B, t_max, dims.Hkv, dims.d), torch.bfloat16)
    _check_list(first, "first", dims.B)
    _check_list(count, "count", dims.B)
    return _done(load_serve_library().lrkv_paged_read(
        ctypes.byref(dims.c()), ctypes.byref(cache.c()), layer, _addr(first), _addr(count), t_max, k_out.data_ptr(),
        v_out.data_ptr(), _stream(stream)), "lrkv_paged_read", check)


def lrkv_paged_attn(dims, cache, layer, q, out, t_q_b=None, score=None, ws=None, stream=None, check=True):
    """out [B,t_q,Hq,d] <- attention of the newest t_q tokens' queries q (bf16) over `layer`'s pages."""
    t_q = q.shape[1]
    for name, t in (("q", q), ("out", out)):
        _check(t, name, (dims.B, t_q, dims.Hq, dims.d), torch.bfloat16)
    _check_list(t_q_b, "t_q_b", dims.B)
    _check_score(score, dims.B, t_q, dims.Hq)
    return _done(load_serve_library().lrkv_paged_attn(
        ctypes.byref(dims.c()), ctypes.byref(cache.c()), layer, q.data_ptr(), t_q, _addr(t_q_b), _ref(score),
        out.data_ptr(), _addr(ws), 0 if ws is None else ws.numel(), _stream(stream)), "lrkv_paged_attn", check)


def lrkv_pages_reserve(dims, cache, t_new, t_new_b=None, stream=None, check=True):
    """Pages for t_new (or t_new_b[b]) more tokens of every sequence."""
    _check_list(t_new_b, "t_new_b", dims.B)
    return _done(load_serve_library().lrkv_pages_reserve(ctypes.byref(dims.c()), ctypes.byref(cache.c()), t_new,
                                                         _addr(t_new_b), _stream(stream)), "lrkv_pages_reserve", check)


def lrkv_pages_advance(dims, cache, t_new, t_new_b=None, stream=None, check=True):
    """seq_len += t_new (or t_new_b)."""
    _check_list(t_new_b, "t_new_b", dims.B)
    return _done(load_serve_library().lrkv_pages_advance(ctypes.byref(dims.c()), ctypes.byref(cache.c()), t_new,
                                                         _addr(t_new_b), _stream(stream)), "lrkv_pages_advance", check)


def _pair(src, dst):
    _check_list(src, "src", src.numel())
    _check_list(dst, "dst", src.numel())
    return src.data_ptr(), dst.data_ptr(), src.numel()


def lrkv_pages_fork(dims, cache, src, dst, ws=None, stream=None, check=True):
    """Sequence dst[i] becomes a copy of sequence src[i] (int32 lists on the device)."""
    s, d, n = _pair(src, dst)
    return _done(load_serve_library().lrkv_pages_fork(
        ctypes.byref(dims.c()), ctypes.byref(cache.c()), s, d, n, _addr(ws), 0 if ws is None else ws.numel(),
        _stream(stream)), "lrkv_pages_fork", check)


def lrkv_pages_free(dims, cache, seqs, stream=None, check=True):
    """Empty the sequences listed in seqs (int32, on the device)."""
    _check_list(seqs, "seqs", seqs.numel())
    return _done(load_serve_library().lrkv_pages_free(ctypes.byref(dims.c()), ctypes.byref(cache.c()),
                                                      seqs.data_ptr(), seqs.numel(), _stream(stream)),
                 "lrkv_pages_free", check)


def lrkv_pages_copy(dims, cache, src, dst, ws=None, stream=None, check=True):
    """Copy pages src[i] to dst[i] (int32 lists on the device) in every layer."""
    s, d, n = _pair(src, dst)
    return _done(load_serve_library().lrkv_pages_copy(
        ctypes.byref(dims.c()), ctypes.byref(cache.c()), s, d, n, _addr(ws), 0 if ws is None else ws.numel(),
        _stream(stream)), "lrkv_pages_copy", check)


def lrkv_pages_compact(dims, cache, ws=None, stream=None, check=True):
    """Move pages so that the live ones have the lowest ids."""
    return _done(load_serve_library().lrkv_pages_compact(ctypes.byref(dims.c()), ctypes.byref(cache.c()), _addr(ws),
                                                         0 if ws is None else ws.numel(), _stream(stream)),
                 "lrkv_pages_compact", check)
