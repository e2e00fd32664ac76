"""Host-side refusals of the prompt, shared-prefix, page and append calls
(no GPU: the library checks its arguments before any launch)."""
import ctypes

import pytest

import long_context_decode_split_gb300 as fd
from long_context_decode_split_gb300 import _build

P = ctypes.c_void_p
A = P(0x10000)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fd.load()


def packed(lib, **kw):
    a = dict(q=A, k=A, v=A, qs=1024, ks=256, vs=256, cq=A, ck=A, B=2, Tq=100, Tk=100, Hq=8, Hkv=2, d=128, scale=0.1,
             causal=1, splits=1, out=A, dt=1, lse=A, ws=None, wsb=0, st=None)
    a.update(kw)
    return lib.fd_prefill_packed(*a.values())


def paged(lib, **kw):
    a = dict(q=A, k=A, v=A, qs=1024, table=A, max_pages=4, num_pages=9, cq=A, lens=A, page=64, B=2, Tq=100, Hq=8,
             Hkv=2, d=128, scale=0.1, causal=1, splits=1, out=A, dt=1, lse=A, ws=None, wsb=0, st=None)
    a.update(kw)
    return lib.fd_prefill_paged(*a.values())


def shared(lib, **kw):
    a = dict(q=A, k=A, v=A, prefix=A, n=2, table=A, max_pages=4, num_pages=9, lens=A, page=64, B=2, Hq=8, Hkv=2, d=128,
             scale=0.1, splits=1, out=A, dt=1, lse=A, ws=A, wsb=1 << 30, st=None)
    a.update(kw)
    return lib.fd_decode_paged_shared_prefix(*a.values())


def dense(lib, **kw):
    a = dict(q=A, kp=A, vp=A, n=100, k=A, v=A, lens=None, B=2, Hq=8, Hkv=2, L=64, d=128, scale=0.1, splits=1, out=A,
             dt=1, lse=A, ws=A, wsb=1 << 30, st=None)
    a.update(kw)
    return lib.fd_decode_dense_shared_prefix(*a.values())


def assign(lib, **kw):
    a = dict(cached=A, new=A, B=2, table=A, max_pages=4, page=64, free=A, nfree=3, head=None, total=5, lens=A, cu=A,
             slots=A, out=A, st=None)
    a.update(kw)
    return lib.fd_assign_pages(*a.values())


def append(lib, **kw):
    a = dict(k=A, v=A, ks=256, vs=256, slots=A, T=3, Hkv=2, d=128, kp=A, vp=A, n=4, page=64, st=None)
    a.update(kw)
    return lib.fd_append_kv_paged(*a.values())


BAD, NO = fd.FD_ERR_INVALID_ARG, fd.FD_ERR_UNSUPPORTED
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kw,want", [
    (dict(d=96), NO), (dict(Hq=18), NO), (dict(Hq=7), BAD), (dict(B=-1), BAD), (dict(Tq=-1), BAD), (dict(Tk=-1), BAD),
    (dict(qs=1016), BAD), (dict(qs=1028), BAD), (dict(ks=128), BAD), (dict(vs=260), BAD), (dict(scale=0.0), BAD),
    (dict(scale=-0.1), BAD), (dict(scale=INF), BAD), (dict(scale=NAN), BAD), (dict(dt=3), BAD), (dict(splits=-1), BAD),
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(out=None), BAD), (dict(cq=None), BAD), (dict(ck=None), BAD),
    (dict(q=P(0x10008)), BAD), (dict(v=P(0x10002)), BAD), (dict(lse=P(0x10002)), BAD),
    (dict(splits=3), fd.FD_ERR_WORKSPACE_TOO_SMALL), (dict(splits=3, ws=A, wsb=100), fd.FD_ERR_WORKSPACE_TOO_SMALL),
    (dict(splits=3, ws=P(0x10004), wsb=1 << 30), BAD), (dict(splits=1 << 20), BAD),
], ids=str)
def test_prefill_packed_refusals(lib, kw, want):
    assert packed(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(page=32), NO), (dict(page=0), BAD), (dict(max_pages=0), BAD), (dict(num_pages=-1), BAD), (dict(table=None), BAD),
    (dict(lens=None), BAD), (dict(k=None), BAD), (dict(cq=None), BAD), (dict(scale=0.0), BAD), (dict(d=80), NO),
    (dict(qs=8), BAD), (dict(num_pages=1 << 27), NO), (dict(splits=2), fd.FD_ERR_WORKSPACE_TOO_SMALL),
    (dict(table=P(0x10002)), BAD),
], ids=str)
def test_prefill_paged_refusals(lib, kw, want):
    assert paged(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(page=16), NO), (dict(n=5), BAD), (dict(n=-1), BAD), (dict(prefix=None), BAD), (dict(table=None), BAD),
    (dict(lens=None), BAD), (dict(scale=-1.0), BAD), (dict(Hq=20), NO), (dict(d=32), NO), (dict(q=None), BAD),
    (dict(k=None), BAD), (dict(out=None), BAD), (dict(num_pages=1 << 27), NO), (dict(dt=9), BAD), (dict(splits=-2), BAD),
    (dict(q=P(0x10004)), BAD),
], ids=str)
def test_shared_prefix_refusals(lib, kw, want):
    assert shared(lib, **kw) == want


def test_shared_prefix_dense_refusals(lib):
    for kw, want in ((dict(n=-1), BAD), (dict(L=-1), BAD), (dict(kp=None), BAD), (dict(k=None), BAD),
                     (dict(scale=0.0), BAD), (dict(d=96), NO), (dict(B=40000, Hq=8, Hkv=8, L=1 << 16), NO)):
        assert dense(lib, **kw) == want, kw


def test_workspace_sizes_with_explicit_chunks(lib):
    assert fd.fd_prefill_workspace_size(2, 100, 8, 2, 4096, 128, 1) == 0
    assert fd.fd_prefill_workspace_size(2, 100, 8, 2, 4096, 128, 3) == 100 * 8 * 3 * 130 * 4 + 256
    assert fd.fd_prefill_num_splits(2, 100, 8, 2, 4096, 128, 3) == 3
    assert fd.fd_prefill_workspace_size(2, 100, 8, 2, 4096, 96, 3) == 0
    with pytest.raises(fd.FdError):
        fd.fd_prefill_num_splits(2, 100, 9, 2, 4096, 128)


@pytest.mark.parametrize("kw,want", [
    (dict(page=128), NO), (dict(B=-1), BAD), (dict(max_pages=0), BAD), (dict(nfree=-1), BAD), (dict(total=-1), BAD),
    (dict(cached=None), BAD), (dict(new=None), BAD), (dict(table=None), BAD), (dict(lens=None), BAD),
    (dict(cu=None), BAD), (dict(out=None), BAD), (dict(slots=None), BAD), (dict(free=None), BAD),
    (dict(slots=P(0x10008)), BAD), (dict(cu=P(0x10002)), BAD),
], ids=str)
def test_assign_refusals(lib, kw, want):
    assert assign(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(page=32), NO), (dict(d=96), NO), (dict(T=-1), BAD), (dict(n=-1), BAD), (dict(Hkv=0), BAD), (dict(ks=120), BAD),
    (dict(vs=257), BAD), (dict(k=None), BAD), (dict(slots=None), BAD), (dict(vp=None), BAD), (dict(k=P(0x10004)), BAD),
    (dict(slots=P(0x10004)), BAD),
], ids=str)
def test_append_refusals(lib, kw, want):
    assert append(lib, **kw) == want


def test_append_fp8_refusals(lib):
    def call(ks=A, vs=A):
        return lib.fd_append_kv_paged_fp8(A, A, 256, 256, A, 3, 2, 128, A, ks, A, vs, 4, 64, None)
    assert call(ks=None) == BAD and call(vs=P(0x10002)) == BAD


def test_out_of_pages_has_a_name(lib):
    assert fd.fd_status_string(fd.FD_ERR_OUT_OF_PAGES).startswith("FD_ERR_OUT_OF_PAGES")
