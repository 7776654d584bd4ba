"""Calls of the serving operators that the other tests do not make: wrong devices, sequences whose
pages ran out, rejected drafts, weights far below the largest one, numbers that are not finite."""
import pytest
import torch

import decode_attention_lrkv_b200 as L
from tests import serve_testutil as U

pytestmark = pytest.mark.gpu
CANARY = 123.0


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("name", L.PagedCache.FIELDS)
def test_a_cache_with_a_tensor_of_the_host_is_refused(name):
    D = L.PagedDims(B=2, Hq=4, Hkv=2, d=128, page=16, n_pages=4, max_pages=2)
    c, ws, one = L.PagedCache(D), L.make_paged_workspace(D), U.ints([0])
    c.__dict__[name] = getattr(c, name).cpu()
    here = torch.cuda.current_stream()
    for kw in ({}, {"stream": here}):
        for call in (lambda: L.lrkv_paged_append(D, c, 0, bf(2, 1, 2, 128), bf(2, 1, 2, 128), **kw),
                     lambda: L.lrkv_paged_read(D, c, 0, None, U.ints([1, 1]), bf(2, 1, 2, 128), bf(2, 1, 2, 128), **kw),
                     lambda: L.lrkv_paged_attn(D, c, 0, bf(2, 1, 4, 128), bf(2, 1, 4, 128), ws=ws, **kw),
                     lambda: L.lrkv_pages_reserve(D, c, 1, **kw), lambda: L.lrkv_pages_advance(D, c, 1, **kw),
                     lambda: L.lrkv_pages_fork(D, c, one, one, ws=ws, **kw), lambda: L.lrkv_pages_free(D, c, one, **kw),
                     lambda: L.lrkv_pages_copy(D, c, one, one, ws=ws, **kw), lambda: L.lrkv_pages_compact(D, c, ws=ws, **kw)):
            with pytest.raises(ValueError, match="CUDA tensor"):
                call()
