"""The paged 4-bit memory's host side: refused arguments launch nothing (no GPU is touched),
sizes are those that rba.h states."""
import ctypes

import pytest

FAKE = 0x10000  # never dereferenced: nothing is launched
I, I64, F, SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from retrieval_block_sparse_b200 import build
    build.build()
    import retrieval_block_sparse_b200 as m
    return m.lib()


def _create(L, buffers=None, **kw):
    from retrieval_block_sparse_b200.rba import _PagedBuffers, _PagedDesc
    d = dict(n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=32, n_pages=64, max_requests=4,
             max_pages=16, dtype=1)
    d.update(kw)
    b = dict(pool=FAKE, rep=FAKE, table=FAKE, lens=FAKE, free_pages=FAKE, n_free=FAKE, status=FAKE)
    b.update(buffers or {})
    h = ctypes.c_void_p()
    s = L.rba_paged_create(ctypes.byref(_PagedDesc(**d)), ctypes.byref(_PagedBuffers(**b)),
                           ctypes.byref(h))
    return s, h


@pytest.fixture
def store(L):
    s, h = _create(L)
    assert s == 0 and h.value
    yield h
    assert L.rba_paged_destroy(h) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(n_q_heads=3), INVALID), (dict(n_kv_heads=0), INVALID), (dict(page_size=0), INVALID),
    (dict(n_pages=0), INVALID), (dict(max_requests=0), INVALID), (dict(max_pages=-1), INVALID),
    (dict(dtype=2), INVALID), (dict(head_dim=130), UNSUPPORTED), (dict(head_dim=98), UNSUPPORTED),
    (dict(max_requests=4097), UNSUPPORTED), (dict(n_pages=1 << 26), UNSUPPORTED),
    (dict(max_pages=1 << 26), UNSUPPORTED)])
def test_create_refuses(L, bad, status):
    s, h = _create(L, **bad)
    assert s == status and not h.value


@pytest.mark.parametrize("name", ["pool", "rep", "table", "lens", "free_pages", "n_free", "status"])
def test_create_wants_every_buffer(L, name):
    assert _create(L, {name: None})[0] == INVALID


def test_create_wants_aligned_pools(L):
    assert _create(L, dict(pool=FAKE + 8))[0] == INVALID
    assert _create(L, dict(rep=FAKE + 4))[0] == INVALID
    assert L.rba_paged_create(None, None, None) == INVALID


def test_sizes(L, store):
    assert [L.rba_paged_strip_bytes(d) for d in (128, 100, 64, 4, 98, 132)] == \
        [2304, 2304, 1152, 1152, -1, -1]
    # 4.5 bits an element
    assert 2304 * 8 / (2 * 16 * 128) == 4.5
    assert L.rba_paged_select_workspace_size(store) == 4 * 2 * 16 * 4
    assert L.rba_paged_attend_workspace_size(store) > 0
    assert L.rba_paged_select_workspace_size(None) == L.rba_paged_attend_workspace_size(None) == 0


def test_extend_and_truncate_refuse(L, store):
    def ext(s=store, new=FAKE, n=4, slots=FAKE, ns=8, starts=FAKE):
        return L.rba_paged_extend(s, new, n, slots, ns, starts, None)
    assert ext(s=None) == ext(new=None) == ext(n=0) == ext(n=5) == ext(slots=None) == \
        ext(ns=-1) == ext(starts=None) == INVALID
    assert L.rba_paged_truncate(store, None, 4, None) == INVALID
    assert L.rba_paged_truncate(None, FAKE, 4, None) == INVALID
    assert L.rba_paged_truncate(store, FAKE, 0, None) == L.rba_paged_truncate(
        store, FAKE, 5, None) == INVALID


def test_append_and_read_refuse(L, store):
    def app(s=store, slots=FAKE, n=4, k=FAKE, v=FAKE):
        return L.rba_paged_append(s, slots, n, k, 256, 128, v, 256, 128, None)
    assert app(s=None) == app(slots=None) == app(n=-1) == app(k=None) == app(v=None) == INVALID
    assert app(n=0, slots=None) == 0

    def rd(s=store, slots=FAKE, n=4, k=FAKE, v=FAKE):
        return L.rba_paged_read(s, slots, n, k, v, None)
    assert rd(s=None) == rd(slots=None) == rd(n=-1) == rd(k=None) == rd(v=None) == INVALID
    assert rd(k=FAKE + 2) == rd(v=FAKE + 8) == INVALID
    assert rd(n=0, slots=None) == 0


def test_select_refuses(L, store):
    def sel(s=store, q=FAKE, n=4, k=3, sink=0, window=0, idx=FAKE, ws=FAKE, nb=1 << 20):
        return L.rba_paged_select(s, q, 1024, 128, n, k, sink, window, idx, ws, nb, None)
    assert sel(s=None) == sel(q=None) == sel(n=0) == sel(n=5) == sel(k=-1) == sel(sink=-1) == \
        sel(window=-1) == sel(idx=None) == sel(ws=None) == INVALID
    assert sel(k=0, idx=None) == 0
    assert sel(nb=4 * 2 * 16 * 4 - 1) == WORKSPACE
    s, h = _create(L, max_pages=20000)
    assert s == 0 and sel(s=h) == UNSUPPORTED  # more candidates than one CTA selects from
    L.rba_paged_destroy(h)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_select_wants_a_workspace_of_floats(L, store, off):
    assert L.rba_paged_select(store, FAKE, 1024, 128, 4, 3, 0, 0, FAKE, FAKE + off, 1 << 20,
                              None) == INVALID


def test_attend_refuses(L, store):
    def att(s=store, q=FAKE, n=4, idx=FAKE, k=3, sink=0, window=0, out=FAKE, ws=FAKE, nb=1 << 30):
        return L.rba_paged_attend(s, q, 1024, 128, n, idx, k, sink, window, F(0.1), out, None, ws,
                                  nb, None)
    assert att(s=None) == att(q=None) == att(n=0) == att(n=5) == att(idx=None) == att(k=-1) == \
        att(sink=-1) == att(window=-1) == att(out=None) == att(ws=None) == INVALID
    assert att(ws=FAKE + 4) == INVALID
    assert att(nb=L.rba_paged_attend_workspace_size(store) - 1) == WORKSPACE
    s, h = _create(L, page_size=1, max_pages=1 << 30, max_requests=2)
    assert s == 0 and att(s=h, n=2, nb=(1 << 62)) == UNSUPPORTED
    L.rba_paged_destroy(h)


def test_step_check_refuses_what_a_steps_calls_would(L, store):
    ws = L.rba_paged_attend_workspace_size(store)

    def chk(s=store, n=4, rows=4, k=3, sink=0, window=0, sel=FAKE, nsel=1 << 20, att=FAKE,
            natt=1 << 30):
        return L.rba_paged_step_check(s, n, rows, k, sink, window, sel, nsel, att, natt)
    assert chk() == chk(rows=0) == chk(k=0, sel=None, nsel=0) == 0
    assert chk(nsel=4 * 2 * 16 * 4, natt=ws) == 0
    assert chk(s=None) == chk(n=0) == chk(n=5) == chk(rows=-1) == chk(k=-1) == chk(sink=-1) == \
        chk(window=-1) == chk(sel=None) == chk(sel=FAKE + 2) == chk(att=None) == \
        chk(att=FAKE + 4) == INVALID
    assert chk(nsel=4 * 2 * 16 * 4 - 1) == chk(natt=ws - 1) == WORKSPACE
    s, h = _create(L, max_pages=20000)
    assert s == 0 and chk(s=h) == UNSUPPORTED
    assert chk(s=h, window=20000 * 32 - 100) == chk(s=h, k=0) == 0  # 4 candidates, none
    L.rba_paged_destroy(h)
    s, h = _create(L, page_size=1, max_pages=1 << 30, max_requests=2)
    assert s == 0 and chk(s=h, n=2, k=0, natt=1 << 62) == UNSUPPORTED
    L.rba_paged_destroy(h)
    s, h = _create(L, n_q_heads=64, n_kv_heads=64)
    big = (1 << 31) - 1
    assert s == 0 and chk(s=h, rows=big) == UNSUPPORTED == L.rba_paged_append(
        h, FAKE, big, FAKE, 8192, 128, FAKE, 8192, 128, None)
    L.rba_paged_destroy(h)


def test_numbers_past_32_bits_are_refused_in_python():
    from retrieval_block_sparse_b200.rba import PagedStore, _fits
    for x in (2 ** 31, 2 ** 32, -2 ** 31 - 1, 2 ** 63):
        with pytest.raises(ValueError):
            _fits(window=x)
    _fits(sink=0, window=2 ** 31 - 1, k=-2 ** 31)
    sizes = dict(n_q_heads=1, n_kv_heads=1, head_dim=64, page_size=16, n_pages=2, max_requests=1,
                 max_pages=2)
    for name in sizes:  # (refused before anything is allocated)
        with pytest.raises(ValueError):
            PagedStore(**{**sizes, name: 2 ** 32 + sizes[name]})


def test_check_wants_a_store(L):
    assert L.rba_paged_check(None, None) == INVALID
