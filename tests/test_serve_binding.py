"""What the Python binding of the serving calls refuses by itself, without a GPU."""
import copy
import os
import pickle
import subprocess
import sys

import pytest
import torch

import decode_attention_lrkv_b200 as L
from decode_attention_lrkv_b200 import build
from decode_attention_lrkv_b200 import serve as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def small(**kw):
    return L.PagedDims(**{**dict(B=2, Hq=4, Hkv=2, d=128, page=16, n_pages=4, max_pages=2), **kw})


def test_a_cache_lies_on_one_device():
    D = small()
    codes = torch.empty(1, 4, 2, 16, 128, dtype=torch.uint8, device="meta")
    table = torch.full((2, 2), -1, dtype=torch.int32)
    for given in (dict(k=codes, page_table=table), dict(page_table=table, v=codes)):
        with pytest.raises(ValueError, match="other tensors are on"):
            L.PagedCache(D, **given)
    c = L.PagedCache(D, device="cpu")
    with pytest.raises(ValueError, match="other tensors are on"):
        c.k = codes
    # and the calls look at each of them
    for name in c.FIELDS:
        mixed = L.PagedCache(D, device="cpu")
        fake = {n: torch.empty_like(getattr(mixed, n), device="meta") for n in c.FIELDS if n != name}
        for t in fake.values():
            t.get_device = lambda: 0
        mixed.__dict__.update(fake)
        with pytest.raises(ValueError, match=f"^{name}: a CUDA tensor on cuda:0 is needed"):
            S._cache_ref(D, mixed, 0)


def test_a_cache_keeps_its_shapes():
    D = small()
    c = L.PagedCache(D, device="cpu")
    for name, bad in (("page_table", torch.zeros(2, 1, dtype=torch.int32)), ("seq_len", torch.zeros(2, dtype=torch.int64)),
                      ("k", c.k[:, :3]), ("scale_v", c.scale_v.transpose(1, 2)), ("refs", torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError, match=name):
            setattr(c, name, bad)
    with pytest.raises(AttributeError, match="dims"):
        c.dims = small(max_pages=9)
    for mine in (1, 2):                                        # what a program adds is its own
        c.mine = mine
    table = torch.full((2, 2), -1, dtype=torch.int32)
    c.page_table = table
    assert c.page_table is table and c.c().page_table == table.data_ptr()
    with pytest.raises(TypeError, match="no keys"):
        L.PagedCache(D, device="cpu", keys=table)
    for other in (copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        assert other.dims == D and all(torch.equal(getattr(other, n), getattr(c, n)) for n in c.FIELDS)


def test_whole_numbers_that_do_not_fit_are_refused(monkeypatch):
    """None of them is cut to 32 bits: 2^32 is no layer 0, and 2^32 + 1 tokens are not one."""
    big = 2 ** 32 + 1
    for name in ("B", "Hq", "Hkv", "n_pages", "max_pages", "n_layers"):
        with pytest.raises(ValueError, match=f"{name}: .* 32 bits"):
            small(**{name: big})
    for kw in (dict(window=big), dict(window=big, slopes=torch.zeros(4))):
        with pytest.raises(ValueError, match="window: .* 32 bits"):
            L.Score(**kw)
    D = small()
    with pytest.raises(ValueError, match="t_q: .* 32 bits"):
        L.lrkv_paged_workspace_size(D, big)
    c = L.PagedCache(D, device="cpu")
    monkeypatch.setattr(S, "_device", lambda t, name: -1)     # as if the host's tensors were on the device
    monkeypatch.setattr(S, "_stream", lambda stream, device: None)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: L.lrkv_paged_append(D, c, big, bf(2, 1, 2, 128), bf(2, 1, 2, 128)),
                 lambda: L.lrkv_paged_read(D, c, big, None, n, bf(2, 1, 2, 128), bf(2, 1, 2, 128)),
                 lambda: L.lrkv_paged_attn(D, c, big, bf(2, 1, 4, 128), bf(2, 1, 4, 128)),
                 lambda: L.lrkv_pages_reserve(D, c, big), lambda: L.lrkv_pages_advance(D, c, big)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


@pytest.mark.parametrize("bad", [torch.zeros(4), torch.zeros(4, dtype=torch.uint8), torch.zeros(0, dtype=torch.int32),
                                 torch.zeros(4, dtype=torch.int64), torch.zeros(2, 2, dtype=torch.int32).T], ids=str)
def test_a_status_word_is_an_int32(bad, monkeypatch):
    monkeypatch.setattr(S, "_device", lambda t, name: -1)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dev_status"):
        L.lrkv_prefill_attn(bf(1, 4, 4, 128), bf(1, 4, 2, 128), bf(1, 4, 2, 128), bf(1, 4, 4, 128), dev_status=bad)


def test_lists_of_sequences_end_where_comparing_them_would_take_long():
    import ctypes
    lib = L.load_serve_library()
    at = 1 << 29                                              # an address that no refused call looks at
    D = small().c()
    C = S._PagedCache(*(at + (i << 24) for i in range(8)))
    D, C = ctypes.byref(D), ctypes.byref(C)
    for n in (2 ** 16 + 1, 2 ** 24):
        assert lib.lrkv_pages_free(D, C, at, n, None) == 2, n
        assert lib.lrkv_pages_fork(D, C, at, at, n, at, 1 << 40, None) == 2, n
    assert lib.lrkv_pages_copy(D, C, at, at, 2 ** 24 + 1, at, 1 << 40, None) == 2


def test_only_a_score_is_taken_for_one(monkeypatch):
    """Dims hold the address of a struct as scores do: they must not be read as one."""
    D = small()
    assert not hasattr(D, "_score_at") and not hasattr(L.Score(), "_at")
    c = L.PagedCache(D, device="cpu")
    monkeypatch.setattr(S, "_device", lambda t, name: -1)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    for bad in (D, 3, "causal"):
        with pytest.raises(TypeError, match="a Score is needed"):
            L.lrkv_paged_attn(D, c, 0, bf(2, 1, 4, 128), bf(2, 1, 4, 128), score=bad)
        with pytest.raises(TypeError, match="a Score is needed"):
            L.lrkv_prefill_attn(bf(1, 4, 4, 128), bf(1, 4, 2, 128), bf(1, 4, 2, 128), bf(1, 4, 4, 128), score=bad)


def run(code):
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT,
                          env={**os.environ, "CUDA_VISIBLE_DEVICES": ""})


@pytest.mark.parametrize("error", ["ImportError('undefined symbol: of_another_torch')", "ModuleNotFoundError('no such file')"])
def test_the_binding_does_without_its_fast_path(error):
    """What keeps _serve_calls from loading is said, and the Python path does the work."""
    r = run(f"""
import sys, warnings
import decode_attention_lrkv_b200 as L
class Broken:
    def find_spec(self, name, path=None, target=None):
        if name.endswith('_serve_calls'):
            raise {error}
sys.meta_path.insert(0, Broken())
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter('always')
    L.load_serve_library()
print('warned:', *[str(x.message) for x in w])
D = L.PagedDims(B=2, Hq=4, Hkv=2, d=128, page=16, n_pages=4, max_pages=2)
print(L.lrkv_paged_workspace_size(D) > 0)
try:
    L.lrkv_pages_reserve(D, L.PagedCache(D, device='cpu'), 1)
except ValueError as e:
    print('refused:', e)
""")
    assert r.returncode == 0, r.stderr
    assert error.split("'")[1] in r.stdout and "True" in r.stdout and "refused: cache" in r.stdout, r.stdout


def test_the_fast_path_is_built_again_for_another_torch(tmp_path, monkeypatch):
    lib, stamp = tmp_path / "_serve_calls.so", tmp_path / "made_for"
    monkeypatch.setattr(build, "CALLS_LIB", str(lib))
    monkeypatch.setattr(build, "CALLS_STAMP", str(stamp))
    assert not build._calls_current()
    lib.write_bytes(b"")
    assert not build._calls_current()
    stamp.write_text(build._calls_made_for())
    assert build._calls_current()
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "9.9")
    assert not build._calls_current()


def test_the_fast_path_that_was_built_is_used():
    build.build()
    S.load_serve_library()
    assert not build._calls_current() or not isinstance(S._calls, S._InPython)


def test_a_failed_build_of_the_fast_path_leaves_the_libraries(tmp_path, monkeypatch):
    lib = tmp_path / "_serve_calls.so"
    lib.write_bytes(b"of another torch")
    monkeypatch.setattr(build, "CALLS_LIB", str(lib))
    monkeypatch.setattr(build, "CALLS_STAMP", str(tmp_path / "made_for"))
    monkeypatch.setattr(build, "CALLS_SRC", str(tmp_path / "missing.cpp"))
    monkeypatch.setattr(build, "_calls_inputs", lambda: [str(lib)])
    with pytest.warns(RuntimeWarning, match="marshals its calls in Python"):
        assert build.build() == build.LIB
    assert not lib.exists()
