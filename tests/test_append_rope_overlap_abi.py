"""The rotating appends refuse pools and scales that overlap another argument
(host-side checks, no GPU)."""
import ctypes

import pytest

import long_context_decode_split_gb300 as fd
from long_context_decode_split_gb300 import _build
from test_diff_rope_abi import Rope

T, HQ, HKV, D, PAGES, B, MAX_POS, ROT = 3, 8, 2, 128, 4, 2, 100, 64
# every buffer in 1 MiB of its own
NAMES = ("q", "k", "v", "slots", "q_out", "kp", "vp", "ks", "vs", "cos_sin", "positions", "cu", "lens", "qw", "kw")
AT = {n: 0x10000000 + 0x100000 * i for i, n in enumerate(NAMES)}


def sizes(fp8, by_offsets):
    pool = PAGES * HKV * 64 * D * (1 if fp8 else 2)
    s = dict(q=T * HQ * D * 2, k=T * HKV * D * 2, v=T * HKV * D * 2, slots=T * 8, q_out=T * HQ * D * 2, kp=pool, vp=pool,
             cos_sin=MAX_POS * ROT * 4, qw=D * 4, kw=D * 4)
    if fp8:
        s["ks"] = s["vs"] = PAGES * HKV * 64 * 4
    if by_offsets:
        s["cu"], s["lens"] = (B + 1) * 4, B * 4
    else:
        s["positions"] = T * 4
    return s


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fd.load()


def call(lib, fp8, by_offsets, at):
    p = {n: ctypes.c_void_p(a) for n, a in at.items()}
    r = Rope(cos_sin=p["cos_sin"], max_pos=MAX_POS, rot=ROT, interleaved=0, halves=0,
             positions=None if by_offsets else p["positions"], cu_seqlens=p["cu"] if by_offsets else None,
             seq_lens=p["lens"] if by_offsets else None, B=B if by_offsets else 0, q_weight=p["qw"], k_weight=p["kw"],
             norm_eps=1e-5)
    head = (p["q"], p["k"], p["v"], HQ * D, HKV * D, HKV * D, p["slots"], T, HQ, HKV, D, ctypes.byref(r), p["q_out"], HQ * D)
    if fp8:
        return lib.fd_append_kv_paged_rope_fp8(*head, p["kp"], p["ks"], p["vp"], p["vs"], PAGES, 64, None)
    return lib.fd_append_kv_paged_rope(*head, p["kp"], p["vp"], PAGES, 64, None)


@pytest.mark.parametrize("by_offsets", [False, True])
@pytest.mark.parametrize("fp8,pool", [(False, "kp"), (False, "vp"), (True, "kp"), (True, "vp"), (True, "ks"), (True, "vs")])
def test_overlaps_are_refused(lib, pool, fp8, by_offsets):
    size = sizes(fp8, by_offsets)
    for other in size:
        if other == pool:
            continue
        # the pool starts with the other buffer, at its last 16 bytes, or ends with its first ones
        for shift in {0, (size[other] - 1) // 16 * 16, -((size[pool] - 1) // 16 * 16)}:
            at = dict(AT)
            at[pool] = AT[other] + shift
            assert call(lib, fp8, by_offsets, at) == fd.FD_ERR_INVALID_ARG, (other, shift)

