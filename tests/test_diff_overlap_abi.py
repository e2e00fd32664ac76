"""The differential calls refuse outputs and workspaces that overlap another
argument (host-side checks, no GPU)."""
import ctypes

import pytest

import long_context_decode_split_gb300 as fd
from long_context_decode_split_gb300 import _build

B, T, HQ, HKV, L, D, PAGES = 2, 100, 8, 2, 256, 128, 9
SPLITS = 2
# every buffer in 4 MiB of its own
NAMES = ("q", "k", "v", "lens", "table", "cu_q", "cu_k", "lam", "weight", "out", "lse", "ws")
AT = {n: 0x10000000 + 0x400000 * i for i, n in enumerate(NAMES)}


def sizes(prompt, paged, f32):
    """Bytes of every buffer of a call."""
    rows = T if prompt else B
    cache = (PAGES * HKV * 64 if paged else T * HKV if prompt else B * HKV * L) * D * 2
    s = dict(q=rows * HQ * D * 2, k=cache, v=cache, lam=rows * HQ * 4, weight=D * 4, out=rows * HQ * D * (4 if f32 else 2),
             lse=rows * HQ * 8, ws=rows * 2 * HQ * SPLITS * (D + 2) * 4 + 256)
    if paged or not prompt:
        s["lens"] = B * 4
    if paged:
        s["table"] = B * 4 * 4
    if prompt:
        s["cu_q"] = (B + 1) * 4
        if not paged:
            s["cu_k"] = (B + 1) * 4
    return s


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fd.load()


def call(lib, prompt, paged, f32, at):
    p = {n: ctypes.c_void_p(a) for n, a in at.items()}
    mix = (p["lam"], HQ, p["weight"], 1e-5)
    tail = (SPLITS, p["out"], 0 if f32 else 1, p["lse"], p["ws"], 1 << 30, None)
    if prompt and paged:
        return lib.fd_prefill_paged_diff(p["q"], p["k"], p["v"], HQ * D, p["table"], 4, PAGES, p["cu_q"], p["lens"], 64, B,
                                         T, HQ, HKV, D, 0.1, 1, *mix, *tail)
    if prompt:
        return lib.fd_prefill_packed_diff(p["q"], p["k"], p["v"], HQ * D, HKV * D, HKV * D, p["cu_q"], p["cu_k"], B, T, T,
                                          HQ, HKV, D, 0.1, 1, *mix, *tail)
    if paged:
        return lib.fd_decode_paged_diff(p["q"], p["k"], p["v"], p["table"], 4, PAGES, p["lens"], 64, B, HQ, HKV, D, 0.1,
                                        *mix, *tail)
    return lib.fd_decode_dense_diff(p["q"], p["k"], p["v"], p["lens"], B, HQ, HKV, L, D, 0.1, *mix, *tail)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("written", ["out", "lse", "ws"])
def test_overlaps_are_refused(lib, written, prompt, paged, f32):
    assert fd.FD_OUT_F32 == 0 and fd.FD_OUT_BF16 == 1
    size = sizes(prompt, paged, f32)
    for other in size:
        if other == written:
            continue
        # `written` starts with the other buffer, at its last 16 bytes, or ends with its first ones
        for shift in {0, (size[other] - 1) // 16 * 16, -((size[written] - 1) // 16 * 16)}:
            at = dict(AT)
            at[written] = AT[other] + shift
            in_place = not prompt and not f32 and (written, other, shift) == ("out", "q", 0)
            if not in_place:
                assert call(lib, prompt, paged, f32, at) == fd.FD_ERR_INVALID_ARG, (other, shift)


def test_prompts_in_place_are_refused(lib):
    """Of one part too, without workspace: a piece may be read twice."""
    for paged in (False, True):
        p = {n: ctypes.c_void_p(a) for n, a in AT.items()}
        mix = (p["lam"], 0, None, 0.0)
        tail = (1, p["q"], 1, None, None, 0, None)
        if paged:
            got = lib.fd_prefill_paged_diff(p["q"], p["k"], p["v"], HQ * D, p["table"], 4, PAGES, p["cu_q"], p["lens"], 64,
                                            B, T, HQ, HKV, D, 0.1, 1, *mix, *tail)
        else:
            got = lib.fd_prefill_packed_diff(p["q"], p["k"], p["v"], HQ * D, HKV * D, HKV * D, p["cu_q"], p["cu_q"], B, T,
                                             T, HQ, HKV, D, 0.1, 1, *mix, *tail)
        assert got == fd.FD_ERR_INVALID_ARG
