"""liblrkv_serve.so without a GPU: its symbols, its refusals, and the binding's."""
import copy
import ctypes
import os
import pickle
import re
import subprocess

import pytest
import torch

import decode_attention_lrkv_b200 as L
from decode_attention_lrkv_b200 import build
from decode_attention_lrkv_b200 import serve as S

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "lrkv_serve.h")
INVALID, UNSUP, ALIGN = 1, 2, 3
FAKE = 0x20000000      # an address that no refused call looks at


@pytest.fixture(scope="module")
def lib():
    build.build()
    return L.load_serve_library()


def test_exports_what_the_header_declares(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"\b(lrkv_[a-z_0-9]+)\s*\(", src))
    out = subprocess.run(["nm", "-D", "--defined-only", L.SERVE_LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert set(re.findall(r"\bT (lrkv_\w+)", out)) == declared
    assert declared == {n for n in S._SIGNATURES}
    assert all(hasattr(L, n) for n in declared)


def _prefill(lib, q=FAKE, k=FAKE, v=FAKE, out=FAKE, q_len=None, kv_len=None, score=None, dims=True, ws=None, ws_bytes=0,
             **kw):
    d = dict(B=2, Hq=8, Hkv=2, d=128, t_q=512, t_k=512)
    d.update({n: kw[n] for n in d if n in kw})
    st = {n: kw.get(n, (512 * h * 128, h * 128, 128)) for n, h in
          (("q_stride", d["Hq"]), ("k_stride", d["Hkv"]), ("v_stride", d["Hkv"]), ("out_stride", d["Hq"]))}
    D = S._PrefillDims(*d.values(), *[x for s in st.values() for x in s])
    return lib.lrkv_prefill_attn(ctypes.byref(D) if dims else None, q, k, v, q_len, kv_len,
                                 ctypes.byref(score) if score else None, out, None, ws, ws_bytes, None)


def test_prefill_refusals(lib):
    assert _prefill(lib, dims=False) == INVALID
    assert _prefill(lib, d=64) == UNSUP
    assert _prefill(lib, Hq=9) == INVALID
    for bad in (dict(B=0), dict(Hkv=0), dict(t_q=-1), dict(t_k=-1), dict(q=None), dict(k=None), dict(v=None),
                dict(out=None), dict(q_stride=(0, 1024, 128)), dict(k_stride=(1 << 20, 256, -128)),
                dict(v_stride=(1 << 20, 260, 128)), dict(out_stride=(1 << 20, 1024, 4))):
        assert _prefill(lib, **bad) == INVALID, bad
    assert _prefill(lib, t_q=1 << 25) == UNSUP
    for bad in ("q", "k", "v", "out", "q_len", "kv_len"):
        assert _prefill(lib, **{bad: FAKE + 8}) == ALIGN, bad
    for bad in (dict(scale=-1.0), dict(scale=float("nan")), dict(softcap=-2.0), dict(softcap=float("inf")),
                dict(softcap=1e-35), dict(window=-1),
                dict(scale=1e10, softcap=1e-25)):
        assert _prefill(lib, score=S._Score(**bad)) == INVALID, bad
    assert _prefill(lib, score=S._Score(slopes=FAKE + 4)) == ALIGN
    assert _prefill(lib, t_q=0) == 0                       # no rows: nothing to do


PTRS = {n: FAKE + 0x1000000 * i for i, n in enumerate(L.PagedCache.FIELDS)}


def _dims(**kw):
    d = dict(B=3, Hq=8, Hkv=2, d=128, page=32, n_pages=64, max_pages=16, n_layers=2, code=0)
    d.update(kw)
    return S._PagedDims(*d.values())


def _cache(**kw):
    return S._PagedCache(*{**PTRS, **kw}.values())


def _calls(lib, D=None, C=None, layer=0, ws=FAKE, ws_bytes=1 << 40, a=FAKE, b=FAKE, lst=None, n=4, score=None):
    """Every paged call with the given arguments: name -> status."""
    D, C = ctypes.byref(D or _dims()), ctypes.byref(C or _cache())
    score = ctypes.byref(score) if score else None
    return {"append": lib.lrkv_paged_append(D, C, layer, a, b, n, lst, None),
            "read": lib.lrkv_paged_read(D, C, layer, None, lst or FAKE, n, a, b, None),
            "attn": lib.lrkv_paged_attn(D, C, layer, a, n, lst, score, b, ws, ws_bytes, None),
            "fork": lib.lrkv_pages_fork(D, C, a, b, n, ws, ws_bytes, None),
            "copy": lib.lrkv_pages_copy(D, C, a, b, n, ws, ws_bytes, None),
            "free": lib.lrkv_pages_free(D, C, a, n, None),
            "reserve": lib.lrkv_pages_reserve(D, C, n, lst, None),
            "advance": lib.lrkv_pages_advance(D, C, n, lst, None),
            "compact": lib.lrkv_pages_compact(D, C, ws, ws_bytes, None)}


def test_paged_refusals(lib):
    for bad in (dict(B=0), dict(Hq=9), dict(Hkv=0), dict(page=24), dict(page=256), dict(n_pages=0), dict(max_pages=0),
                dict(n_layers=0), dict(code=2)):
        assert set(_calls(lib, D=_dims(**bad)).values()) == {INVALID}, bad
    for bad in (dict(d=64), dict(Hq=18), dict(max_pages=1 << 20)):
        assert set(_calls(lib, D=_dims(**bad)).values()) == {UNSUP}, bad
    for field in L.PagedCache.FIELDS:
        assert set(_calls(lib, C=_cache(**{field: None})).values()) == {INVALID}, field
        assert set(_calls(lib, C=_cache(**{field: FAKE + 4})).values()) == {ALIGN}, field
    for bad in (-1, 2):
        got = _calls(lib, layer=bad, ws=None)               # the page calls take no layer; stop them by other means
        assert got["append"] == got["read"] == got["attn"] == INVALID


def test_paged_argument_refusals(lib):
    D, C = ctypes.byref(_dims()), ctypes.byref(_cache())
    A = FAKE
    assert lib.lrkv_paged_append(D, C, 0, None, A, 1, None, None) == INVALID
    assert lib.lrkv_paged_append(D, C, 0, A, A, -1, None, None) == INVALID
    assert lib.lrkv_paged_append(D, C, 0, A, A + 2, 1, None, None) == ALIGN
    assert lib.lrkv_paged_append(D, C, 0, A, A, 1, A + 4, None) == ALIGN
    assert lib.lrkv_paged_append(D, C, 0, A, A, 0, None, None) == 0
    assert lib.lrkv_paged_read(D, C, 0, None, None, 1, A, A, None) == INVALID
    assert lib.lrkv_paged_read(D, C, 0, A + 4, A, 1, A, A, None) == ALIGN
    assert lib.lrkv_paged_read(D, C, 0, None, A, 0, A, A, None) == 0
    size = lib.lrkv_paged_workspace_size(D, 4)
    assert size > 0 and size % 256 == 0
    assert lib.lrkv_paged_workspace_size(None, 1) == lib.lrkv_paged_workspace_size(D, 0) == 0
    assert lib.lrkv_paged_workspace_size(D, 65) == 0
    attn = lambda t_q=4, q=A, out=A, t_q_b=None, score=None, ws=A, n=size: lib.lrkv_paged_attn(
        D, C, 0, q, t_q, t_q_b, score, out, ws, n, None)
    assert attn(q=None) == attn(out=None) == attn(ws=None) == attn(t_q=0) == attn(n=size - 1) == INVALID
    assert attn(t_q=65) == UNSUP
    assert attn(q=A + 8) == attn(out=A + 2) == attn(t_q_b=A + 4) == attn(ws=A + 8) == ALIGN
    assert attn(score=ctypes.byref(S._Score(window=-3))) == INVALID
    for call in (lib.lrkv_pages_fork, lib.lrkv_pages_copy):
        assert call(D, C, A, A, -1, A, size, None) == call(D, C, None, A, 1, A, size, None) == INVALID
        assert call(D, C, A, A, 1, None, size, None) == call(D, C, A, A, 1, A, 256, None) == INVALID
        assert call(D, C, A, A + 4, 1, A, size, None) == ALIGN
        assert call(D, C, None, None, 0, A, size, None) == 0
    assert lib.lrkv_pages_free(D, C, None, 1, None) == lib.lrkv_pages_free(D, C, A, -1, None) == INVALID
    assert lib.lrkv_pages_free(D, C, None, 0, None) == 0
    assert lib.lrkv_pages_compact(D, C, A, 256, None) == lib.lrkv_pages_compact(D, C, None, size, None) == INVALID
    assert lib.lrkv_pages_reserve(D, C, -1, None, None) == lib.lrkv_pages_advance(D, C, -1, None, None) == INVALID
    assert lib.lrkv_pages_reserve(D, C, 0, None, None) == 0
    # tile numbers and tensor coordinates are 32-bit
    wide = _dims(B=60000, Hq=32, Hkv=8, max_pages=1 << 17)
    assert lib.lrkv_paged_attn(ctypes.byref(wide), C, 0, A, 1, None, None, A, A, 1 << 40, None) == UNSUP
    deep = _dims(Hq=32, Hkv=8, n_pages=1 << 22, n_layers=4)
    assert lib.lrkv_paged_attn(ctypes.byref(deep), C, 0, A, 1, None, None, A, A, 1 << 40, None) == UNSUP


def test_a_workspace_serves_fewer_rows_too(lib):
    for kw in (dict(Hq=8, Hkv=2), dict(Hq=16, Hkv=2), dict(Hq=6, Hkv=2), dict(max_pages=4), dict(max_pages=1 << 18)):
        D = _dims(**kw)
        sizes = [lib.lrkv_paged_workspace_size(ctypes.byref(D), t) for t in range(1, 65)]
        assert sizes == sorted(sizes), kw


def test_binding_refuses_what_the_library_cannot_see(lib):
    D = L.PagedDims(B=2, Hq=4, Hkv=2, d=128, page=16, n_pages=4, max_pages=2)
    cache = L.PagedCache(D, device="cpu")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):          # tensors of the host
        L.lrkv_paged_append(D, cache, 0, bf(2, 1, 2, 128), bf(2, 1, 2, 128))
    with pytest.raises(ValueError, match="CUDA"):
        L.lrkv_pages_reserve(D, cache, 1)
    with pytest.raises(ValueError):
        L.lrkv_prefill_attn(bf(1, 4, 4, 128).float(), bf(1, 4, 2, 128), bf(1, 4, 2, 128), bf(1, 4, 4, 128))
    with pytest.raises(ValueError, match="CUDA"):
        L.lrkv_prefill_attn(bf(1, 4, 4, 128), bf(1, 4, 2, 128), bf(1, 4, 2, 128), bf(1, 4, 4, 128))
    with pytest.raises(TypeError):
        L.PagedCache(D, device="cpu", keys=bf(1))
    with pytest.raises(ValueError, match="page_table"):
        L.PagedCache(D, device="cpu", page_table=torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="invalid dims"):
        L.make_paged_workspace(D, 65, device="cpu")
    assert cache.page_table.tolist() == [[-1, -1], [-1, -1]] and int(cache.refs.sum()) == 0


def test_dims_and_scores_can_be_copied():
    D = L.PagedDims(B=2, Hq=4, Hkv=2, d=128, page=16, n_pages=4, max_pages=2)
    for other in (copy.deepcopy(D), pickle.loads(pickle.dumps(D))):
        assert other == D and bytes(other.c()) == bytes(D.c())
    s = L.Score(softcap=3.0, window=5)
    assert copy.deepcopy(s) == s and pickle.loads(pickle.dumps(s)) == s
