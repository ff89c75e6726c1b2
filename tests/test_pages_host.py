"""The paged-cache calls on the CPU: what the library refuses before it
launches anything, what the binding refuses before it calls the library, and
the index functions that the kernels apply to lengths, starts, table entries
and slots (compiled for the host from the kernels' own header)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20          # an aligned address that no refused call follows


@pytest.fixture(scope="module")
def skv():
    from lossless_kv_cache_amd import skv as m
    if not os.path.exists(m.LIB_PATH):
        from lossless_kv_cache_amd import build
        build.build()
    m.lib()
    return m


def pool(skv, dtype=None, layers=1, pages=10, page_tokens=16, heads=8, dim=128, strides=None, abi=1):
    st = (0, page_tokens * heads * dim, heads * dim, dim) if strides is None else strides
    return skv._PAGES.pack(abi, skv.BF16 if dtype is None else dtype, layers, pages, page_tokens, heads, dim, 0, *st)


def rows(skv, dtype=None, tokens=4, strides=(0, 1024, 128)):
    return skv._ROWS.pack(skv.BF16 if dtype is None else dtype, tokens, *strides)


def plan(skv, requests=4, width=8, stride=8, free=A, n_free=4, page_tokens=16, tokens=4, lens=A, starts=A, slots=A):
    return skv.lib().skv_page_plan(lens, A, requests, A, width, stride, free, n_free, page_tokens, tokens, slots, A,
                                   starts, A, None, None)


def test_plan_refusals(skv):
    assert plan(skv, lens=None) == skv.ERR_ARG
    assert plan(skv, starts=None) == skv.ERR_ARG
    assert plan(skv, slots=None) == skv.ERR_ARG
    assert plan(skv, stride=7) == skv.ERR_ARG
    for kw in (dict(requests=0), dict(requests=4097), dict(width=0), dict(page_tokens=0), dict(page_tokens=4),
               dict(page_tokens=24), dict(page_tokens=2048), dict(width=1 << 27, stride=1 << 27),
               dict(tokens=1 << 31)):
        assert plan(skv, **kw) == skv.ERR_SHAPE, kw


@pytest.mark.parametrize("name", ["skv_page_write", "skv_page_read"])
def test_rows_refusals(skv, name):
    call = getattr(skv.lib(), name)

    def go(pg=None, rw=None, kp=A, vp=A, k=A, v=A, slots=A, ks=None, vs=None):
        return call(pool(skv) if pg is None else pg, kp, vp, rows(skv) if rw is None else rw, k, v, slots, ks, vs, None,
                    None)

    for kw in (dict(kp=None), dict(vp=None), dict(k=None), dict(slots=None), dict(kp=A + 8), dict(v=A + 2),
               dict(ks=A), dict(vs=A), dict(pg=pool(skv, strides=(0, 16 * 1024, 1024, 130))),
               dict(pg=pool(skv, strides=(0, 16 * 1024, 1028, 128))), dict(pg=pool(skv, strides=(0, 4, 1024, 128))),
               dict(pg=pool(skv, layers=2, strides=(4, 16 * 1024, 1024, 128))),
               dict(rw=rows(skv, strides=(0, 1026, 128))), dict(rw=rows(skv, strides=(0, 1024, 4)))):
        assert go(**kw) == skv.ERR_ARG, kw
    E, B = skv.E4M3, skv.BF16
    for kw in (dict(pg=pool(skv, abi=2)), dict(pg=pool(skv, dtype=skv.INT16)), dict(pg=pool(skv, page_tokens=12)),
               dict(pg=pool(skv, pages=0)), dict(pg=pool(skv, heads=0)), dict(pg=pool(skv, dim=8)),
               dict(pg=pool(skv, dim=0)), dict(pg=pool(skv, heads=1024)), dict(pg=pool(skv, layers=0)),
               dict(pg=pool(skv, pages=1 << 27)), dict(rw=rows(skv, dtype=E)), dict(rw=rows(skv, dtype=skv.INT16)),
               dict(rw=rows(skv, tokens=1 << 31))):
        assert go(**kw) == skv.ERR_SHAPE, kw
    # e4m3 rows of e4m3 pages are copies: 16-byte strides are 16 elements, and no scale
    assert go(pg=pool(skv, dtype=E), rw=rows(skv, dtype=E, strides=(0, 1032, 128))) == skv.ERR_ARG
    assert go(pg=pool(skv, dtype=E), rw=rows(skv, dtype=E), ks=A) == skv.ERR_ARG
    # no rows: nothing to do
    assert go(rw=rows(skv, dtype=B, tokens=0), k=None, v=None, slots=None) == skv.OK


def attention(skv, requests=2, tokens=2, q_heads=32, width=8, most=1, causal=1, scale=0.1, ts=8, q_st=(4096, 128),
              o_st=(4096, 128), q=A, table=A, lens=A, starts=0, ks=0, vs=0, out=A, abi=1):
    return skv._ATTENTION.pack(abi, requests, tokens, q_heads, width, most, causal, scale, ts, *q_st, *o_st, q, A, A,
                               table, lens, starts, ks, vs, out, 0, 0)


def test_attention_refusals(skv):
    def go(pg=None, work=None, size=0, **kw):
        n = ctypes.c_size_t(size)
        return skv.lib().skv_page_attention(pool(skv) if pg is None else pg, attention(skv, **kw), work,
                                            ctypes.byref(n), None), n.value

    rc, need = go()
    assert rc == skv.OK and need >= 256
    for kw in (dict(causal=2), dict(scale=float("nan")), dict(tokens=3), dict(ks=A), dict(vs=A), dict(ts=7),
               dict(q=A + 8), dict(out=A + 2), dict(q=0), dict(out=0), dict(table=0), dict(lens=0),
               dict(q_st=(4100, 128)), dict(o_st=(4096, 129)), dict(pg=pool(skv, strides=(0, 16384, 1024, 4)))):
        assert go(**kw)[0] == skv.ERR_ARG, kw
    for kw in (dict(abi=2), dict(requests=0), dict(requests=65536, tokens=65536), dict(width=0), dict(q_heads=0),
               dict(q_heads=20), dict(q_heads=8 * 65), dict(tokens=1 << 27, starts=A), dict(width=1 << 27, ts=1 << 27),
               dict(width=(1 << 26) + 1, ts=1 << 27),
               dict(pg=pool(skv, layers=2)), dict(pg=pool(skv, dim=96)), dict(pg=pool(skv, dtype=skv.INT16))):
        assert go(**kw)[0] == skv.ERR_SHAPE, kw
    # a workspace too small is refused with the size needed, one out of line as an argument
    assert go(work=A, size=need - 1) == (skv.ERR_CAPACITY, need)
    assert go(work=A + 4, size=need)[0] == skv.ERR_ARG
    # a batch without rows has nothing to do
    assert go(work=A, size=1 << 40, tokens=0, starts=A, q=0, out=0)[0] == skv.OK
    assert skv.lib().skv_page_check(None, None, None) == skv.ERR_ARG


def test_binding_refuses_host_tensors(skv):
    i = torch.zeros(4, dtype=torch.int32)
    t = torch.zeros((4, 8), dtype=torch.int32)
    pages = torch.zeros((10, 16, 8, 128), dtype=torch.bfloat16)
    kv = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    q = torch.zeros((4, 32, 128), dtype=torch.bfloat16)
    for call in (lambda: skv.page_plan(i, i, t, i, 16, 4), lambda: skv.page_write(kv, kv, pages, pages, i),
                 lambda: skv.page_read(pages, pages, i), lambda: skv.page_attention(q, pages, pages, t, i),
                 lambda: skv.page_check(i), lambda: skv.PageCache(skv.INT16, 1, 4, 16, 8, 128, device="cpu"),
                 lambda: skv.PageCache(skv.BF16, 1, 4, 16, 8, 128, device="cpu", k_scale=torch.ones((1, 8)))):
        with pytest.raises(ValueError):
            call()
    e = skv.SkvError(skv.ERR_PAGES, "x")
    assert "out of range" in str(e) and e.status == -9


# ------------------------------------------------------------------ the kernels' index functions on the host
@pytest.fixture(scope="module")
def index(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not installed")
    so = str(tmp_path_factory.mktemp("index") / "index.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror",
                    os.path.join(ROOT, "tests", "host", "pages_index.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    L.pages.restype = ctypes.c_uint32
    L.slot.restype = ctypes.c_int32
    L.span.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.c_int64] + [ctypes.c_uint32] * 4 + [ctypes.c_void_p]
    return L


def test_plan_requests(index):
    def req(*a):
        o, n = ctypes.c_uint32(), ctypes.c_uint32()
        bad = index.plan(*a, ctypes.byref(o), ctypes.byref(n))
        return bad, o.value, n.value

    assert req(10, 3, 8, 4) == (0, 7, 10)
    assert req(0, 0, 8, 4) == (0, 0, 0)
    assert req(128, 128, 8, 4) == (0, 0, 128)
    top = (1 << 31) - 1
    assert req(top, 1, 1 << 28, 3) == (0, top - 1, top)
    for a in ((10, -1, 8, 4), (-1, 0, 8, 4), (3, 4, 8, 4), (129, 1, 8, 4), (-(1 << 31), -(1 << 31), 8, 4)):
        assert req(*a) == (1, 0, 0), a
    assert [index.pages(n, 4) for n in (0, 1, 16, 17)] == [0, 1, 1, 2]
    assert index.pages(0xFFFFFFFF, 3) == 1 << 29


def test_slots_and_pages(index):
    assert index.slot(3, 5, 4) == 53
    assert index.slot(0, 0, 3) == 0
    assert index.slot(-1, 0, 4) == -1 and index.slot(-(1 << 31), 7, 4) == -1
    assert index.slot((1 << 31) - 1, 0, 3) == -1 and index.slot((1 << 28) - 1, 0, 3) == -1
    assert index.slot((1 << 28) - 2, 7, 3) == ((1 << 28) - 2) * 8 + 7
    out = ctypes.c_uint32(9)
    for entry, count, want, bad in ((0, 1, 0, 0), (9, 10, 9, 0), (10, 10, 0, 1), (-1, 10, 0, 1),
                                    (-(1 << 31), 1 << 30, 0, 1), ((1 << 31) - 1, 10, 0, 1)):
        assert index.page(entry, count, ctypes.byref(out)) == bad and out.value == want


def test_spans(index):
    def span(*a):
        out = (ctypes.c_uint32 * 3)()
        return index.span(*a, out), tuple(out)

    # len, r0, r1, tokens, width, page_shift, max_new
    assert span(100, 5, 9, 20, 8, 4, 4) == (0, (5, 4, 100))
    assert span(0, 5, 5, 20, 8, 4, 4) == (0, (5, 0, 0))
    assert span(2, 0, 9, 20, 8, 4, 9) == (0, (0, 9, 2))          # more queries than tokens: the first see nothing
    assert span(100, 5, 10, 20, 8, 4, 4) == (2, (0, 0, 0))
    for a in ((-1, 0, 1, 20, 8, 4, 4), (129, 0, 1, 20, 8, 4, 4), (10, -1, 1, 20, 8, 4, 4), (10, 3, 2, 20, 8, 4, 4),
              (10, 19, 21, 20, 8, 4, 4), (10, 1 << 31, (1 << 31) + 1, 20, 8, 4, 4)):
        assert span(*a) == (1, (0, 0, 0)), a
