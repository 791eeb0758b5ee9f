"""Paged-cache entry points without a GPU: layout queries and refusals (every check
runs on the host before anything is launched)."""
import ctypes as C

import pytest
import torch

from long_context_decoding_eta_b200 import _lib as L
from long_context_decoding_eta_b200 import paged

DIMS = L.Dims.of(3, 8, 2, 128, 64, 640)
FAKE = C.c_void_p(4096)                     # aligned, never dereferenced by a refused call
ODD = C.c_void_p(4100)
BIG = C.c_size_t(1 << 40)


def _d(dims):
    return C.byref(dims)


def test_state_layout():
    # header 8, lengths 3 -> 4, table 30 -> 32, ref 13 -> 16, free list 13 -> 16
    assert L.eta_page_state_offsets(DIMS, 13) == (0, 8, 12, 44, 60)
    assert L.eta_page_state_words(DIMS, 13) == 76
    assert L.eta_page_workspace_size(DIMS, 13) >= 4 * (2 * 4 + 3 + 3 * 13)


@pytest.mark.parametrize("dims,n_pages,code", [
    (L.Dims.of(3, 8, 2, 96, 64, 640), 13, 2), (L.Dims.of(3, 8, 2, 128, 32, 640), 13, 2),
    (L.Dims.of(3, 8, 2, 128, 64, 650), 13, 2), (L.Dims.of(3, 6, 2, 128, 64, 640), 13, 2),
    (L.Dims.of(3, 8, 3, 128, 64, 640), 13, 1), (L.Dims.of(0, 8, 2, 128, 64, 640), 13, 1),
    (DIMS, 0, 1), (DIMS, -4, 1), (DIMS, 1 << 24, 2)])
def test_refused_sizes(dims, n_pages, code):
    lib = L.lib()
    assert L.eta_page_state_words(dims, n_pages) == 0
    assert L.eta_page_workspace_size(dims, n_pages) == 0
    with pytest.raises(L.EtaError) as e:
        L.eta_page_state_offsets(dims, n_pages)
    assert e.value.code == code
    n = C.c_int32(n_pages)
    assert lib.eta_page_init(_d(dims), n, FAKE, None) == code
    assert lib.eta_page_append(_d(dims), n, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, FAKE, BIG,
                               None, None) == code
    assert lib.eta_page_fork(_d(dims), n, FAKE, FAKE, FAKE, FAKE, FAKE, 1, FAKE, BIG, None,
                             None) == code
    assert lib.eta_page_free(_d(dims), n, FAKE, FAKE, 1, FAKE, BIG, None, None) == code
    assert lib.eta_page_compact(_d(dims), n, FAKE, FAKE, FAKE, FAKE, BIG, None, None) == code
    assert lib.eta_page_copy(_d(dims), n, FAKE, FAKE, FAKE, FAKE, 1, FAKE, BIG, None,
                             None) == code
    assert lib.eta_paged_build_block_meta(_d(dims), n, FAKE, FAKE, FAKE, FAKE, 0, -1, 0, FAKE,
                                          FAKE, FAKE, FAKE, None, None, None, None) == code
    assert lib.eta_paged_decode(_d(dims), n, FAKE, None, FAKE, FAKE, FAKE, FAKE, None, None, 0.0,
                                0.0, 0, None, None, 0, FAKE, FAKE, FAKE, BIG, None, None) == code
    assert lib.eta_shared_decode(_d(dims), n, 1, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                 0.0, 0.0, 0, FAKE, FAKE, FAKE, BIG, None, None) == code


def _page_call(name, state=FAKE, K=FAKE, V=FAKE, x=FAKE, ws=FAKE, size=BIG, n=1):
    """One page operation with arguments that it refuses (a call that would launch is
    never made here: the pointers are not memory)."""
    lib, d = L.lib(), _d(DIMS)
    return dict(
        append=lambda: lib.eta_page_append(d, 13, state, K, V, x, x, x, n, ws, size, None, None),
        fork=lambda: lib.eta_page_fork(d, 13, state, K, V, x, x, n, ws, size, None, None),
        free=lambda: lib.eta_page_free(d, 13, state, x, n, ws, size, None, None),
        copy=lambda: lib.eta_page_copy(d, 13, K, V, x, x, n, ws, size, None, None),
        compact=lambda: lib.eta_page_compact(d, 13, state, K, V, ws, size, None, None))[name]()


@pytest.mark.parametrize("name", ["append", "fork", "free", "copy", "compact"])
def test_page_calls_refuse_their_arguments(name):
    if name != "copy":
        assert _page_call(name, state=None) == _page_call(name, state=ODD) == 1
    if name != "free":
        for kw in (dict(K=None), dict(V=None), dict(K=ODD), dict(V=ODD)):
            assert _page_call(name, **kw) == 1, kw
    small = C.c_size_t(L.eta_page_workspace_size(DIMS, 13) - 1)
    for kw in (dict(ws=None), dict(ws=ODD), dict(size=small)):
        assert _page_call(name, **kw) == 3, kw
    if name != "compact":
        assert _page_call(name, x=None) == 1
        assert _page_call(name, n=-1) == 1
        assert _page_call(name, n=0) == 0           # nothing to do, nothing launched
    if name in ("fork", "free"):
        assert _page_call(name, n=4) == 1           # more than B


def test_paged_decode_refuses_its_arguments():
    lib, d = L.lib(), _d(DIMS)

    def call(q=FAKE, tau=FAKE, K=FAKE, V=FAKE, table=FAKE, lens=FAKE, idx=FAKE, cnt=FAKE, T=0.0,
             prune=0, vsum=None, bcnt=None, fmt=0, o=FAKE, lse=FAKE, ws=FAKE, size=BIG):
        return lib.eta_paged_decode(d, 13, q, tau, K, V, table, lens, idx, cnt, T, 0.0, prune,
                                    vsum, bcnt, fmt, o, lse, ws, size, None, None)

    for name in ("q", "K", "V", "table", "lens", "o", "lse"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "K", "V"):
        assert call(**{name: ODD}) == 1, name
    assert call(cnt=None) == 1              # a block list without its lengths
    assert call(fmt=2) == 1 and call(prune=3) == 1
    assert call(T=-0.5) == 1 and call(T=float("nan")) == 1 and call(T=float("inf")) == 1
    assert call(prune=1) == 1               # FLOOR without the block sums
    assert call(prune=1, idx=None, vsum=FAKE, bcnt=FAKE) == 1
    assert call(ws=None) == 3 and call(ws=ODD) == 3 and call(size=C.c_size_t(64)) == 3


def test_shared_decode_refuses_its_arguments():
    lib, d = L.lib(), _d(DIMS)

    def call(n=2, q=FAKE, tau=FAKE, K=FAKE, V=FAKE, table=FAKE, lens=FAKE, off=FAKE, pre=FAKE,
             T=0.0, fmt=0, o=FAKE, lse=FAKE, ws=FAKE, size=BIG):
        return lib.eta_shared_decode(d, 13, n, q, tau, K, V, table, lens, off, pre, T, 0.0, fmt,
                                     o, lse, ws, size, None, None)

    for name in ("q", "K", "V", "table", "lens", "off", "pre", "o", "lse"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "K", "V", "o"):
        assert call(**{name: ODD}) == 1, name
    assert call(fmt=2) == 1 and call(n=0) == 1 and call(n=4) == 1
    assert call(T=-1.0) == 1 and call(T=float("nan")) == 1
    assert call(ws=None) == 3 and call(ws=ODD) == 3 and call(size=C.c_size_t(64)) == 3
    assert L.eta_shared_decode_workspace_size(DIMS, 0) == 0
    assert L.eta_shared_decode_workspace_size(DIMS, 4) == 0
    assert L.eta_shared_decode_workspace_size(DIMS, 3) > 0


def test_status_words():
    assert L.eta_status_from_device(L.DEVSTAT_NO_PAGE) == 8
    assert L.eta_status_from_device(L.DEVSTAT_BAD_ROW) == 1
    assert L.eta_status_from_device(L.DEVSTAT_BAD_ROW | L.DEVSTAT_TIMEOUT) == 5
    assert L.eta_status_string(8) == "page pool exhausted"


def test_python_layer_refuses_host_tensors_and_shapes():
    k = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        paged.PagedKVCache(2, 2, 64, 64, 4, 4, K=k, V=k)
    with pytest.raises(ValueError, match="together"):
        paged.PagedKVCache(2, 2, 64, 64, 4, 4, K=k)
