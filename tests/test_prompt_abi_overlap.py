"""fd_assign_pages refuses buffers that overlap (host-side checks, no GPU)."""
import ctypes

import pytest

import long_context_decode_split_gb300 as fd
from long_context_decode_split_gb300 import _build

# every buffer in a 4 KiB page of its own: B = 8, max_pages = 4, 16 free pages, 10 slots
NAMES = ("cached", "new", "table", "free", "head", "lens", "cu", "slots", "head_out")
AT = {n: 0x100000 + 0x1000 * i for i, n in enumerate(NAMES)}
SIZE = dict(cached=32, new=32, table=128, free=64, head=4, lens=32, cu=36, slots=80, head_out=4)
OUTPUTS = ("table", "lens", "cu", "slots", "head_out")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fd.load()


def assign(lib, at):
    p = {n: ctypes.c_void_p(a) for n, a in at.items()}
    return lib.fd_assign_pages(p["cached"], p["new"], 8, p["table"], 4, 64, p["free"], 16, p["head"], 10, p["lens"],
                               p["cu"], p["slots"], p["head_out"], None)


@pytest.mark.parametrize("other", NAMES)
@pytest.mark.parametrize("out", OUTPUTS)
def test_overlapping_buffers_are_refused(lib, out, other):
    if out == other:
        return
    # `out` starts at the other buffer, at its last element, or ends with its first one (slots are 16-byte aligned)
    step = 16 if "slots" in (out, other) else 4
    last = (SIZE[other] - 4) // step * step
    before = (SIZE[out] - 4) // step * step
    for shift in {0, last, -before}:
        if shift == 0 and (out, other) in (("lens", "cached"), ("head_out", "head")):
            continue  # in place
        at = dict(AT)
        at[out] = AT[other] + shift
        assert assign(lib, at) == fd.FD_ERR_INVALID_ARG, shift
    # in place over an input that holds something else too
    at = dict(AT, lens=AT["cached"], new=AT["cached"])
    assert assign(lib, at) == fd.FD_ERR_INVALID_ARG
