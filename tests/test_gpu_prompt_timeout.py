"""The time-out path of the prompt rows' pipeline waits, without faulting the GPU.

The test-only hook shortens every wait to 1 ms and makes the copy warp withhold
the keys of one block: no copy and no arrival, so nothing is in flight for that
stage.  Every role's wait runs out in turn; the kernel records
FD_ERR_DEVICE_TIMEOUT, lets its copies land, frees its tensor memory and
returns.  A normal call afterwards has to be right (also on the same SMs: the
tensor memory is free again), and a 1 ms limit alone must not fire.
"""
import math
import time

import pytest
import torch

from rows_reference import attend64, check_rows, gather_pages, generator, limits, offsets, randn, random_pool

pytestmark = pytest.mark.gpu


def packed(fd, T, G, d=128):
    g = generator(T)
    q, k, v = randn(g, T, 2 * G, d), randn(g, T, 2, d), randn(g, T, 2, d)

    def call():
        return fd.fd_prefill_packed(q, k, v, offsets([T]))

    def check():
        out, lse = call()
        check_rows(out, lse, attend64(q, k, v, limits(T, T, True), 1 / math.sqrt(d)))
    return call, check


def shared(fd, B, skip, d=128):
    g = generator(B)
    lens = [skip * 64 + 70 + b for b in range(B)]
    kp, vp, table, pool = random_pool(lens, 2, d, g, skip=skip)
    q = randn(g, B, 8, d)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    prefix = table[0, :skip].clone()

    def call():
        return fd.fd_decode_paged_shared_prefix(q, kp, vp, prefix, table, pool, sl, num_splits=2)

    def check():
        out, lse = call()
        for b, n in enumerate(lens):
            k, v = gather_pages(kp, table[b], n), gather_pages(vp, table[b], n)
            check_rows(out[b:b + 1], lse[b:b + 1], attend64(q[b:b + 1], k, v, torch.tensor([n]), 1 / math.sqrt(d)))
    return call, check


CASES = {
    "two tiles": lambda fd: packed(fd, 700, 4),     # more tokens than a tile: two tiles per CTA
    "one tile": lambda fd: shared(fd, 5, 20),       # fewer: a single tile, two pipelines
    "two tiles, pages": lambda fd: shared(fd, 40, 20),
    "one tile, packed": lambda fd: packed(fd, 30, 2, 64),
}


@pytest.mark.parametrize("tile", [0, 1, 2, 3])
@pytest.mark.parametrize("case", CASES)
def test_withheld_keys_time_out_and_are_reported(fd, case, tile):
    call, check = CASES[case](fd)
    if case == "one tile, packed" and tile > 0:
        tile = 0  # 30 keys are one block
    check()
    assert fd.fd_device_status(clear=True) == fd.FD_OK
    try:
        fd.fd_debug_inject_wait_timeout(1_000_000, tile)
        t0 = time.time()
        call()
        status = fd.fd_device_status(clear=True)
        elapsed = time.time() - t0
    finally:
        fd.fd_debug_inject_wait_timeout(0, -1)
    assert status == fd.FD_ERR_DEVICE_TIMEOUT
    assert elapsed < 5.0, elapsed
    for _ in range(3):
        check()
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_short_limit_alone_does_not_fire(fd):
    calls = [packed(fd, 12000, 4)[0], shared(fd, 40, 500)[0], shared(fd, 3, 500)[0]]
    try:
        fd.fd_debug_inject_wait_timeout(1_000_000, -1)
        for call in calls:
            call()
        assert fd.fd_device_status(clear=True) == fd.FD_OK
    finally:
        fd.fd_debug_inject_wait_timeout(0, -1)
