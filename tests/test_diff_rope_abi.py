"""Host-side refusals of the rotation, rotating append and differential calls
(no GPU: the library checks its arguments before any launch)."""
import ctypes

import pytest

import long_context_decode_split_gb300 as fd
from long_context_decode_split_gb300 import _build

P = ctypes.c_void_p
A = P(0x10000)
BAD, NO, SMALL = fd.FD_ERR_INVALID_ARG, fd.FD_ERR_UNSUPPORTED, fd.FD_ERR_WORKSPACE_TOO_SMALL
INF, NAN = float("inf"), float("nan")


class Rope(ctypes.Structure):
    """fd_rope of include/fd.h."""
    _fields_ = [("cos_sin", P), ("max_pos", ctypes.c_int), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("halves", ctypes.c_int), ("positions", P), ("cu_seqlens", P), ("seq_lens", P), ("B", ctypes.c_int),
                ("q_weight", P), ("k_weight", P), ("norm_eps", ctypes.c_float)]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fd.load()


def at(page):
    """Addresses a megabyte apart."""
    return P(0x1000000 + 0x100000 * page)


# T = 3 tokens, 8 and 2 heads of 128: rows of 2048 and 512 bytes
Q, K, V, QO, KO, TABLE, POOL, SLOTS = (at(i) for i in range(8))


def rope_of(kw):
    r = dict(cos_sin=TABLE, max_pos=100, rot=64, interleaved=0, halves=0, positions=A, cu_seqlens=None, seq_lens=None,
             B=0, q_weight=None, k_weight=None, norm_eps=1e-5)
    r.update({n: kw.pop(n) for n in list(kw) if n in r})
    return Rope(**r)


def norm_rope(lib, **kw):
    r = rope_of(kw)
    a = dict(q=Q, k=K, qs=1024, ks=256, T=3, Hq=8, Hkv=2, d=128, rope=ctypes.byref(r), qo=QO, ko=KO, qos=1024, kos=256,
             st=None)
    a.update(kw)
    return lib.fd_norm_rope(*a.values())


def append(lib, **kw):
    r = rope_of(kw)
    a = dict(q=Q, k=K, v=V, qs=1024, ks=256, vs=256, slots=SLOTS, T=3, Hq=8, Hkv=2, d=128, rope=ctypes.byref(r), qo=QO,
             qos=1024, kp=POOL, vp=at(9), n=4, page=64, st=None)
    a.update(kw)
    return lib.fd_append_kv_paged_rope(*a.values())


ROPE_BAD = [
    (dict(cos_sin=None), BAD), (dict(max_pos=0), BAD), (dict(rot=0), BAD), (dict(rot=136), BAD), (dict(rot=24), NO),
    (dict(rot=80, halves=1), BAD), (dict(positions=None), BAD), (dict(positions=None, cu_seqlens=A, B=2), BAD),
    (dict(B=-1), BAD), (dict(q_weight=A, norm_eps=0.0), BAD), (dict(k_weight=A, norm_eps=NAN), BAD),
    (dict(k_weight=A, norm_eps=INF), BAD), (dict(q_weight=P(0x10008)), BAD), (dict(cos_sin=P(0x10004)), BAD),
    (dict(positions=P(0x10002)), BAD), (dict(rope=None), BAD), (dict(T=-1), BAD), (dict(Hq=-1), BAD), (dict(d=96), NO),
    (dict(qs=1016), BAD), (dict(qs=1028), BAD), (dict(ks=128), BAD), (dict(qos=8), BAD), (dict(q=None), BAD),
    (dict(k=None), BAD), (dict(qo=None), BAD), (dict(q=P(0x10008)), BAD), (dict(qo=P(0x10002)), BAD),
    (dict(qo=P(Q.value + 16)), BAD), (dict(qo=P(Q.value + 2048)), BAD), (dict(qo=Q, qos=2048), BAD), (dict(qo=K), BAD),
    (dict(qo=P(TABLE.value + 25584)), BAD), (dict(positions=P(QO.value + 4)), BAD),
    (dict(positions=None, cu_seqlens=P(QO.value + 16), seq_lens=A, B=2), BAD),
]


@pytest.mark.parametrize("kw,want", ROPE_BAD + [
    (dict(ko=None), BAD), (dict(ko=Q), BAD), (dict(ko=QO), BAD), (dict(ko=P(K.value + 512)), BAD),
    (dict(Hq=0, Hkv=0), BAD), (dict(kos=100), BAD), (dict(T=1 << 28, Hq=64, qs=8192, qos=8192), NO),
    # slices of one row: the queries' columns run into the keys'
    (dict(k=P(Q.value + 1024), qs=2048, ks=2048, qo=Q, qos=2048), BAD),
], ids=str)
def test_norm_rope_refusals(lib, kw, want):
    assert norm_rope(lib, **dict(kw)) == want


@pytest.mark.parametrize("kw,want", ROPE_BAD + [
    (dict(page=32), NO), (dict(page=0), BAD), (dict(n=-1), BAD), (dict(Hkv=0), BAD), (dict(v=None), BAD),
    (dict(vs=200), BAD), (dict(slots=None), BAD), (dict(slots=P(0x10004)), BAD), (dict(kp=None), BAD),
    (dict(vp=None), BAD), (dict(vp=P(0x10008)), BAD), (dict(qo=V), BAD), (dict(qo=P(POOL.value + 16)), BAD),
], ids=str)
def test_append_refusals(lib, kw, want):
    assert append(lib, **dict(kw)) == want


def test_append_fp8_needs_its_scales(lib):
    r = rope_of({})

    def call(ks=A, vs=A):
        return lib.fd_append_kv_paged_rope_fp8(Q, K, V, 1024, 256, 256, SLOTS, 3, 8, 2, 128, ctypes.byref(r), QO, 1024,
                                               POOL, ks, at(9), vs, 4, 64, None)
    assert call(ks=None) == BAD and call(vs=None) == BAD and call(ks=P(0x10002)) == BAD


def test_nothing_to_do_is_fine(lib):
    assert norm_rope(lib, T=0, q=None, k=None, qo=None, ko=None, cos_sin=None, positions=None) == fd.FD_OK
    assert append(lib, T=0, q=None, k=None, v=None, qo=None, slots=None, kp=None, vp=None, n=0) == fd.FD_OK


MIX = dict(lam=A, ls=0, w=None, eps=1e-5)


def dense(lib, **kw):
    a = dict(q=A, k=A, v=A, lens=None, B=2, Hq=8, Hkv=2, L=256, d=128, scale=0.1, **MIX, splits=1, out=A, dt=1, lse=A,
             ws=None, wsb=0, st=None)
    a.update(kw)
    return lib.fd_decode_dense_diff(*a.values())


def paged(lib, **kw):
    a = dict(q=A, k=A, v=A, table=A, max_pages=4, num_pages=9, lens=A, page=64, B=2, Hq=8, Hkv=2, d=128, scale=0.1,
             **MIX, splits=1, out=A, dt=1, lse=A, ws=None, wsb=0, st=None)
    a.update(kw)
    return lib.fd_decode_paged_diff(*a.values())


def packed_rows(lib, **kw):
    a = dict(q=A, k=A, v=A, qs=1024, ks=256, vs=256, cq=A, ck=A, B=2, Tq=100, Tk=100, Hq=8, Hkv=2, d=128, scale=0.1,
             causal=1, **MIX, splits=1, out=A, dt=1, lse=A, ws=None, wsb=0, st=None)
    a.update(kw)
    return lib.fd_prefill_packed_diff(*a.values())


def paged_rows(lib, **kw):
    a = dict(q=A, k=A, v=A, qs=1024, table=A, max_pages=4, num_pages=9, cq=A, lens=A, page=64, B=2, Tq=100, Hq=8,
             Hkv=2, d=128, scale=0.1, causal=1, **MIX, splits=1, out=A, dt=1, lse=A, ws=None, wsb=0, st=None)
    a.update(kw)
    return lib.fd_prefill_paged_diff(*a.values())


@pytest.mark.parametrize("call", [dense, paged, packed_rows, paged_rows])
@pytest.mark.parametrize("kw,want", [
    (dict(d=96), NO), (dict(Hq=18), NO), (dict(Hq=7), BAD), (dict(B=-1), BAD), (dict(scale=0.0), BAD),
    (dict(scale=-1.0), BAD), (dict(scale=INF), BAD), (dict(scale=NAN), BAD), (dict(lam=None), BAD), (dict(ls=7), BAD),
    (dict(ls=-8), BAD), (dict(lam=P(0x10002)), BAD), (dict(w=P(0x10004)), BAD), (dict(w=A, eps=0.0), BAD),
    (dict(w=A, eps=NAN), BAD), (dict(w=A, eps=-1.0), BAD), (dict(splits=-1), BAD), (dict(dt=7), BAD), (dict(q=None), BAD),
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(out=None), BAD), (dict(q=P(0x10008)), BAD), (dict(out=P(0x10008)), BAD),
    (dict(lse=P(0x10002)), BAD), (dict(splits=3), SMALL), (dict(splits=3, ws=A, wsb=100), SMALL),
    (dict(splits=3, ws=P(0x10004), wsb=1 << 30), BAD),
], ids=str)
def test_diff_refusals(lib, call, kw, want):
    assert call(lib, **kw) == want


@pytest.mark.parametrize("call,kw,want", [
    (dense, dict(L=-1), BAD), (dense, dict(B=40000, Hq=8, Hkv=8, L=1 << 16), NO), (dense, dict(lens=P(0x10002)), BAD),
    (paged, dict(page=16), NO), (paged, dict(page=0), BAD), (paged, dict(table=None), BAD), (paged, dict(lens=None), BAD),
    (paged, dict(max_pages=0), BAD), (paged, dict(num_pages=-1), BAD), (paged, dict(num_pages=1 << 27), NO),
    (paged, dict(table=P(0x10002)), BAD),
    (packed_rows, dict(qs=1016), BAD), (packed_rows, dict(ks=128), BAD), (packed_rows, dict(Tk=-1), BAD),
    (packed_rows, dict(cq=None), BAD), (packed_rows, dict(ck=None), BAD), (packed_rows, dict(splits=1 << 20), BAD),
    (paged_rows, dict(page=32), NO), (paged_rows, dict(table=None), BAD), (paged_rows, dict(lens=None), BAD),
    (paged_rows, dict(qs=8), BAD), (paged_rows, dict(num_pages=1 << 27), NO),
], ids=str)
def test_more_diff_refusals(lib, call, kw, want):
    assert call(lib, **kw) == want


def test_diff_workspace_sizes_with_explicit_chunks(lib):
    assert fd.fd_num_splits_diff(2, 8, 2, 1000, 128, 3) == 3
    assert fd.fd_decode_diff_workspace_size(2, 8, 2, 1000, 64, 1) == 0
    assert fd.fd_decode_diff_workspace_size(2, 8, 2, 1000, 64, 3) == 2 * 16 * 3 * (64 + 2) * 4 + 256
    assert fd.fd_prefill_diff_num_splits(2, 100, 8, 2, 4096, 128, 3) == 3
    assert fd.fd_prefill_diff_workspace_size(2, 100, 8, 2, 4096, 128, 3) == 100 * 16 * 3 * 130 * 4 + 256
    assert fd.fd_prefill_diff_workspace_size(2, 100, 8, 2, 4096, 96, 3) == 0
    for f, args in ((fd.fd_num_splits_diff, (1, 9, 2, 64, 128)), (fd.fd_prefill_diff_num_splits, (1, 9, 9, 2, 64, 128))):
        with pytest.raises(fd.FdError):
            f(*args)


def test_nothing_to_attend_is_fine(lib):
    assert dense(lib, B=0, q=None, out=None, lam=None) == fd.FD_OK
    assert packed_rows(lib, Tq=0, q=None, out=None, lam=None) == fd.FD_OK
